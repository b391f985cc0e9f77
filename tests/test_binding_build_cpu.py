"""The compiled binding is built anew for another torch, and refused by one that it was not built for."""
import os
import shutil

import pytest
import torch

import exact_tiled_attention_38_b200 as eta
from exact_tiled_attention_38_b200 import build as eta_build


def test_key_is_that_of_the_torch_in_use():
    version, abi = eta_build.torch_build(eta_build.torch_dir())
    assert version == torch.__version__ and abi == int(torch._C._GLIBCXX_USE_CXX11_ABI)
    assert eta_build.torch_dir() == os.path.dirname(torch.__file__)


def test_another_torch_builds_it_anew(tmp_path):
    eta_build.build_binding()
    version, abi = eta_build.torch_build(eta_build.torch_dir())
    assert eta_build.binding_up_to_date(eta_build.binding_key(version, abi))
    assert not eta_build.binding_up_to_date(eta_build.binding_key(version + "1", abi))
    assert not eta_build.binding_up_to_date(eta_build.binding_key(version, 1 - abi))
    copy = tmp_path / "old.so"
    shutil.copy(eta_build.BINDING_OUT, copy)
    os.utime(copy, (0, 0))  # older than its sources
    assert not eta_build.binding_up_to_date(eta_build.binding_key(version, abi), str(copy))
    assert not eta_build.binding_up_to_date(eta_build.binding_key(version, abi), str(tmp_path / "none.so"))


def test_a_binding_for_another_torch_is_refused():
    assert eta.attn_paged  # this one's own is taken
    from exact_tiled_attention_38_b200 import paged

    key = eta_build.binding_key(torch.__version__, torch._C._GLIBCXX_USE_CXX11_ABI)
    assert paged._binding.built_for == key
    with pytest.raises(RuntimeError, match="build"):
        paged._check_build(key.replace("torch ", "torch 9"))


def test_what_torchs_files_say(tmp_path):
    (tmp_path / "version.py").write_text("nothing")
    with pytest.raises(RuntimeError, match="version.py"):
        eta_build.torch_build(str(tmp_path))
    (tmp_path / "version.py").write_text("__version__ = '1.2.3+cu1'\n")
    assert eta_build.torch_build(str(tmp_path)) == ("1.2.3+cu1", 1)
    config = tmp_path / "share" / "cmake" / "Torch"
    config.mkdir(parents=True)
    (config / "TorchConfig.cmake").write_text('set(TORCH_CXX_FLAGS "-D_GLIBCXX_USE_CXX11_ABI=0")\n')
    assert eta_build.torch_build(str(tmp_path)) == ("1.2.3+cu1", 0)


def test_no_sources_are_needed_to_run(tmp_path):
    """The package's Python files and built libraries are enough."""
    import subprocess
    import sys

    eta_build.build()
    pkg = os.path.dirname(eta.__file__)
    to = tmp_path / os.path.basename(pkg)
    to.mkdir()
    for f in os.listdir(pkg):
        if f.endswith((".py", ".so")) and f != "build.py":
            shutil.copy(os.path.join(pkg, f), to)
    code = ("import exact_tiled_attention_38_b200 as e, os; assert os.path.dirname(e.__file__) == os.environ['AT']; "
            "print(e.attn_rope_turns(8)[1], e.attn_paged.__name__)")
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={**os.environ, "PYTHONPATH": str(tmp_path), "AT": str(to)})
    assert out.returncode == 0 and out.stdout.split() == ["1.0", "attn_paged"], out.stderr
