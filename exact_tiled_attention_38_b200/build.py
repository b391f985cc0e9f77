"""Build the CUDA library in-tree: ``libattn.so`` next to this file, and the
compiled part of the Python binding, ``_binding.so`` (where torch is installed,
whose tensors it takes; the library itself needs neither).

Compiled for sm_100a only (B200). Usage: ``python -m exact_tiled_attention_38_b200.build``.
"""
from __future__ import annotations

import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

from . import _binding_key as binding_key

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
SRC = os.path.join(PKG_DIR, "csrc", "attn_lib.cu")
OUT = os.path.join(PKG_DIR, "libattn.so")
# Every source the library is compiled from: all of csrc/ and the header.
DEPS = sorted(
    os.path.join(PKG_DIR, "csrc", f)
    for f in os.listdir(os.path.join(PKG_DIR, "csrc"))
    if f.endswith((".cu", ".cuh", ".h"))
) + [os.path.join(ROOT, "include", "attn.h")]

BINDING_SRC = os.path.join(PKG_DIR, "csrc", "binding.cpp")
BINDING_OUT = os.path.join(PKG_DIR, "_binding.so")
BINDING_DEPS = [BINDING_SRC, os.path.join(ROOT, "include", "attn.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared",
]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date(out: str = OUT, deps=None) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(d) <= t for d in (DEPS if deps is None else deps))


def torch_dir():
    """Where torch is installed (found, not imported), or None."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else list(spec.submodule_search_locations)[0]


def torch_build(torch: str):
    """(version, C++ ABI) of the torch installed there, from its own files. Where they do
    not name the ABI it is the C++11 one, the only one that current builds have."""
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"__version__ = '([^']+)'", f.read())
    if version is None:
        raise RuntimeError("version.py of torch does not say which one it is")
    config, abi = os.path.join(torch, "share", "cmake", "Torch", "TorchConfig.cmake"), None
    if os.path.exists(config):
        with open(config) as f:
            abi = re.search(r"_GLIBCXX_USE_CXX11_ABI=([01])", f.read())
    return version.group(1), int(abi.group(1)) if abi else 1


def binding_up_to_date(key: str, out: str = BINDING_OUT) -> bool:
    if not up_to_date(out, BINDING_DEPS):
        return False
    with open(out, "rb") as f:
        return key.encode() in f.read()


def build_binding(force: bool = False, verbose: bool = False):
    """``_binding.so`` against the installed torch; None where there is none. Built anew
    where the one there is older than its sources or was built for another torch."""
    torch = torch_dir()
    if torch is None:
        return None
    version, abi = torch_build(torch)
    key = binding_key(version, abi)
    if not force and binding_up_to_date(key):
        return BINDING_OUT
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = os.path.join(torch, "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wextra",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", f'-DETA_BINDING_KEY="{key}"', "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-o", BINDING_OUT + ".tmp", BINDING_SRC, "-L", os.path.join(torch, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    if res.stderr:
        print(res.stderr, file=sys.stderr)  # (warnings)
    os.replace(BINDING_OUT + ".tmp", BINDING_OUT)
    return BINDING_OUT


def build(force: bool = False, verbose: bool = False) -> str:
    build_binding(force, verbose)
    if not force and up_to_date():
        return OUT
    cmd = [nvcc_path(), *NVCC_FLAGS, "-o", OUT + ".tmp", SRC]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(OUT + ".tmp", OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
