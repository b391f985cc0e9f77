"""Python binding of the paged-cache operators (``include/attn.h``): attention of
new tokens over a paged cache, rotary positions and their append to the cache,
page update and compaction. The package offers them under its own name.

Argument marshalling only, as in the rest of the binding, but in a compiled
module (``csrc/binding.cpp``): a serving step makes these calls back to back.
There is no fallback; without the module every call raises.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch  # (the compiled module needs its libraries)

from . import _D, _F, AttnError, _binding_key, _check, _stream_handle, load_library

try:
    from . import _binding
except ImportError as e:
    raise RuntimeError("the compiled binding is not built, or not for this torch; run "
                       "`python -m exact_tiled_attention_38_b200.build`") from e


def _check_build(built_for):
    key = _binding_key(torch.__version__, torch._C._GLIBCXX_USE_CXX11_ABI)
    if built_for != key:
        raise RuntimeError(f"the compiled binding is another one's ({built_for} here is {key}); run "
                           "`python -m exact_tiled_attention_38_b200.build`")


_check_build(_binding.built_for)


def _init():
    lib = load_library()
    _binding.init(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in (
        "attn_paged", "attn_paged_f16", "attn_rope", "attn_rope_f16", "attn_rope_append",
        "attn_rope_append_f16", "attn_pages_update", "attn_pages_compact")))


_init()


def _stream(stream):
    """None (the tensors' device's current stream) or a handle as a whole number."""
    return None if stream is None else _stream_handle(stream) or 0


def _done(result, name):
    if type(result) is int:
        raise AttnError(result, name)
    return result


def attn_paged(q, kpages, vpages, table, cu_q, kv_lens, max_q: Optional[int] = None,
               window: int = 0, scale: Optional[float] = None, o=None, lse=None, stream=None,
               want_lse: bool = True) -> Tuple:
    """Attention of new tokens over a paged cache (chunked prefill, decode, or a mix).

    q [total, Hq, d] (bf16 or fp16; rows may be parts of wider ones), pools
    [num_pages, Hkv, page_size, d], table [B, width], cu_q [B + 1] and kv_lens [B]
    int32: sequence b's new tokens are rows cu_q[b]:cu_q[b + 1] of q, the last of
    its kv_lens[b] cached positions, causal, with a sliding window if given.
    max_q bounds the new tokens of any sequence; the default, total, is slower where
    they are few (give 1 for a decode batch). Returns (o [total, Hq, d],
    lse [total, Hq]). Runs ``attn_paged`` / ``attn_paged_f16``.
    """
    return _done(_binding.paged(q, kpages, vpages, table, cu_q, kv_lens, max_q, window, scale, o,
                                lse, want_lse, _stream(stream)), "attn_paged")


def attn_rope_turns(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                    low: float = 1.0, high: Optional[float] = None, original: float = 4096.0):
    """Turns per position of each rotary pair (float64, on the CPU) and the amplitude.

    scaling: "none", "linear", "base", "parts" (high defaults to 32) or "bands"
    (high defaults to 4); see ``attn_rope_turns`` in include/attn.h.
    """
    names = ("none", "linear", "base", "parts", "bands")
    if scaling not in names:
        raise ValueError(f"scaling must be one of {names}")
    if high is None:
        high = 32.0 if scaling == "parts" else 4.0
    buf = (_D * max(rot // 2, 1))()
    amp = _F(0.0)
    code = load_library().attn_rope_turns(buf, ctypes.byref(amp), int(rot), float(base),
                                          names.index(scaling), float(factor), float(low),
                                          float(high), float(original))
    _check(code, "attn_rope_turns")
    return torch.tensor(list(buf), dtype=torch.float64), amp.value


class _Rope(torch.autograd.Function):
    """The rotation in an autograd graph: linear, with the rotation back as its gradient
    (whose own gradient is the rotation again)."""

    @staticmethod
    def forward(ctx, q, k, pos, turns, amp, interleaved, back, name):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(pos, turns)
        ctx.how = amp, interleaved, not back, name
        return _done(_binding.rope(q, k, pos, turns, amp, interleaved, None, None, back, None), name)

    @staticmethod
    def backward(ctx, *grads):
        out = [None] * 8
        asked = [i for i in (0, 1) if grads[i] is not None and ctx.needs_input_grad[i]]
        if asked:
            x = [_plain(grads[i]) for i in asked] + [None]
            for i, g in zip(asked, _Rope.apply(x[0], x[1], *ctx.saved_tensors, *ctx.how)):
                out[i] = g
        return tuple(out)


def _plain(g):
    """g as the operator takes it: d innermost, strides of whole 16-byte units."""
    n, s = g.shape, g.stride()
    fits = s[3] == 1 and not any(t % 8 for t, m in zip(s[:3], n) if m > 1) and g.data_ptr() % 16 == 0
    return g if fits else g.clone(memory_format=torch.contiguous_format)


def _rope(q, k, pos, turns, amp, interleaved, q_out, k_out, back, stream, name):
    stream = _stream(stream)
    if not (torch.is_grad_enabled() and any(isinstance(x, torch.Tensor) and x.is_cuda and x.requires_grad
                                            for x in (q, k, q_out, k_out))):
        return _done(_binding.rope(q, k, pos, turns, amp, interleaved, q_out, k_out, back, stream), name)
    if q_out is not None or k_out is not None:
        raise ValueError("an output cannot be given where a gradient is recorded "
                         "(under torch.no_grad() it can)")
    args = (q, k, pos, turns, amp, interleaved, back, name)
    if stream is None:
        return _Rope.apply(*args)
    # Current while the graph is recorded, so that the gradient runs on it too.
    here, dev = torch.cuda.current_stream(q.device), q.device
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, dev) if stream else torch.cuda.default_stream(dev)):
        out = _Rope.apply(*args)
    for t in out:
        if t is not None:
            t.record_stream(here)
    return out


def attn_rope(q, k, pos, turns, amp: float = 1.0, interleaved: bool = False, q_out=None,
              k_out=None, stream=None) -> Tuple:
    """Rotary positions of q [B, Hq, N, d] and k [B, Hkv, N, d] (or None), bf16 or fp16.

    Any strides with d innermost; an output may be its input, and is laid out
    like it if none is given. pos int32 [N] or [B, N]; turns and amp from
    ``attn_rope_turns`` (turns on q's device): the first 2 * len(turns) values of
    each head are rotated. Returns (q_out, k_out). Where q or k requires a
    gradient it is recorded, and no output can be given. (The library's attention
    records none: for a gradient through it, bring your own.)
    """
    return _rope(q, k, pos, turns, amp, interleaved, q_out, k_out, False, stream, "attn_rope")


def attn_rope_bwd(dq, dk, pos, turns, amp: float = 1.0, interleaved: bool = False, dq_in=None,
                  dk_in=None, stream=None) -> Tuple:
    """Gradients of ``attn_rope``'s inputs from those of its outputs (same arguments)."""
    return _rope(dq, dk, pos, turns, amp, interleaved, dq_in, dk_in, True, stream, "attn_rope_bwd")


def attn_rope_append(q, k, v, kpages, vpages, table, cu_q, kv_lens, turns, amp: float = 1.0,
                     interleaved: bool = False, pos=None, q_out=None, stream=None):
    """Rotate new tokens' q and k, and put k and v into the paged cache, in one pass.

    q [total, Hq, d], k and v [total, Hkv, d] (rows may be parts of wider ones, as
    one projection gives them); cache arguments as in ``attn_paged``. Positions
    are the tokens' places in the cache unless pos (int32 [total]) is given.
    Returns q_out; the pools are updated in place.
    """
    return _done(_binding.append(q, k, v, kpages, vpages, table, cu_q, kv_lens, turns, amp,
                                 interleaved, pos, q_out, _stream(stream)), "attn_rope_append")


def attn_pages_update(kpages, vpages, table, lens, refs, source, add, table_out=None,
                      lens_out=None, refs_out=None, info=None, stream=None) -> Tuple:
    """One step of the cache's bookkeeping: row b of the next state goes on from
    row source[b] (-1: from nothing) and grows by add[b] tokens; shared last pages
    are copied in every layer. Pools [layers, num_pages, Hkv, page_size, d] or one
    layer's; table [B, width], lens, source, add [B], refs [num_pages], int32.
    Returns (table, lens, refs, info) of the next state; info [2] is zero, or the
    pages that were missing and the rows that outgrew the table (nothing changed
    then). See ``attn_pages_update`` in include/attn.h.
    """
    return _done(_binding.update(kpages, vpages, table, lens, refs, source, add, table_out, lens_out,
                                 refs_out, info, _stream(stream)), "attn_pages_update")


def attn_pages_compact(kpages, vpages, table, lens, refs, table_out=None, refs_out=None, info=None,
                       stream=None) -> Tuple:
    """Move the live pages to the lowest indices, in every layer, with the fewest copies.

    Arguments as in ``attn_pages_update``. Returns (table, refs, info) of the next
    state; info [2]: live pages, moved pages. Pages held from outside move too: with
    n = (refs > 0).sum() of the counts before, the k-th of those at n and above is
    now the k-th page that was free below n (a holder with a row of its own in the
    table need not ask).
    """
    return _done(_binding.compact(kpages, vpages, table, lens, refs, table_out, refs_out, info,
                                  _stream(stream)), "attn_pages_compact")
