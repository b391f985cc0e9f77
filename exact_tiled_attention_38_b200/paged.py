"""Python binding of the paged-cache operators (``include/attn.h``): attention of
new tokens over a paged cache, rotary positions and their append to the cache,
page update and compaction. The package offers them under its own name.

Argument marshalling only, as in the rest of the binding. A decode step makes
these calls every few microseconds, so their checks are kept cheap: identities
instead of comparisons, shapes taken once, no context switch when the tensors'
device is the current one.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _D, _F, _L, ATTN_OK, AttnError, _check, _Pages, _stream_handle, load_library

_BF16, _F16, _F32, _F64, _I32 = (torch.bfloat16, torch.float16, torch.float32, torch.float64,
                                 torch.int32)
_empty, _empty_like = torch.empty, torch.empty_like


def _call(fn, index, stream, *args):
    """Run entry point `fn` with `args` and a stream on device `index`."""
    f = getattr(load_library(), fn)
    if index == torch.cuda.current_device():
        code = f(*args, _raw_stream(index) if stream is None else _stream_handle(stream))
    else:
        with torch.cuda.device(index):
            code = f(*args, _raw_stream(index) if stream is None else _stream_handle(stream))
    if code != ATTN_OK:
        raise AttnError(code, fn)


# The current stream's handle without the Stream object around it (about a
# microsecond a call), where torch offers it.
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(index):
    if _current_raw is not None:
        return _current_raw(index) or None
    return torch.cuda.current_stream(index).cuda_stream or None


def _int32(t, name, index, shape):
    if t.dtype is not _I32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on cuda:{index}")
    return t.data_ptr()


def _cache(kpages, vpages, table):
    """(_Pages, device index, layers, layer_stride) of pools [num_pages, Hkv, page_size, d],
    or [layers, num_pages, Hkv, page_size, d], in any strides with d innermost."""
    dtype, index = kpages.dtype, kpages.get_device()
    if dtype is not _BF16 and dtype is not _F16:
        raise ValueError("kpages and vpages must be bf16 or fp16")
    if not kpages.is_cuda:
        raise ValueError("kpages must be a CUDA tensor")
    shape, strides = kpages.shape, kpages.stride()
    if vpages.dtype is not dtype or vpages.shape != shape or vpages.stride() != strides or \
            vpages.get_device() != index:
        raise ValueError("vpages must have kpages' type, device, shape and strides")
    layers, layer_stride = 0, 0
    if len(shape) == 5:
        layers, layer_stride = shape[0], strides[0]
        shape, strides = shape[1:], strides[1:]
    if len(shape) != 4 or strides[3] != 1:
        raise ValueError("kpages must be [num_pages, Hkv, page_size, d] (or with layers in front), "
                         "d innermost")
    rows = table.shape
    if table.dtype is not _I32 or len(rows) != 2 or table.get_device() != index or \
            not table.is_contiguous():
        raise ValueError(f"table must be a contiguous int32 tensor [B, width] on cuda:{index}")
    P, Hkv, page, d = shape
    stride, head, token, _ = strides
    # A dimension of one element has no stride that matters: give it the packed one.
    if page <= 1:
        token = d
    if Hkv <= 1:
        head = page * d
    if P <= 1:
        stride = max(Hkv * page * d, 8)
    return (_Pages(kpages.data_ptr(), vpages.data_ptr(), table.data_ptr(), stride, head, token, P,
                   page, rows[1], Hkv, d), index, layers, layer_stride, rows[0])


def _packed(t, name, dtype, index, heads, d):
    """(shape, token stride) of a packed tensor [total, heads, d] whose rows may be
    parts of wider ones."""
    shape = t.shape
    if t.dtype is not dtype or len(shape) != 3 or t.get_device() != index:
        raise ValueError(f"{name} must be a 3-D {dtype} tensor [tokens, heads, d] on cuda:{index}")
    n, h, c = shape
    if c != d or (heads is not None and h != heads):
        raise ValueError(f"{name} must have {heads if heads is not None else 'its'} heads of {d}")
    s = t.stride()
    if (s[2] != 1 and d > 1) or (s[1] != d and h > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return shape, (s[0] if n > 1 else h * d)


def attn_paged(q, kpages, vpages, table, cu_q, kv_lens, max_q: Optional[int] = None,
               window: int = 0, scale: Optional[float] = None, o=None, lse=None, stream=None,
               want_lse: bool = True) -> Tuple:
    """Attention of new tokens over a paged cache (chunked prefill, decode, or a mix).

    q [total, Hq, d] (bf16 or fp16; rows may be parts of wider ones), pools
    [num_pages, Hkv, page_size, d], table [B, width], cu_q [B + 1] and kv_lens [B]
    int32: sequence b's new tokens are rows cu_q[b]:cu_q[b + 1] of q, the last of
    its kv_lens[b] cached positions, causal, with a sliding window if given.
    max_q bounds the new tokens of any sequence (default: total). Returns
    (o [total, Hq, d], lse [total, Hq]). Runs ``attn_paged`` / ``attn_paged_f16``.
    """
    cache, index, layers, _, B = _cache(kpages, vpages, table)
    if layers:
        raise ValueError("kpages must be one layer's pool [num_pages, Hkv, page_size, d]")
    dtype = kpages.dtype
    shape, stride = _packed(q, "q", dtype, index, None, cache.d)
    total, Hq, d = shape
    cu_p = _int32(cu_q, "cu_q", index, (B + 1,))
    len_p = _int32(kv_lens, "kv_lens", index, (B,))
    if o is None:
        o = _empty(shape, device=q.device, dtype=dtype)
    elif o.dtype is not dtype or o.get_device() != index or o.shape != shape or \
            not o.is_contiguous():
        raise ValueError("o must be a contiguous tensor of q's shape, type and device")
    if lse is None:
        if want_lse:
            lse = _empty((total, Hq), device=q.device, dtype=_F32)
    elif lse.dtype is not _F32 or lse.get_device() != index or lse.shape != (total, Hq) or \
            not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [total, Hq] on q's device")
    _call("attn_paged_f16" if dtype is _F16 else "attn_paged", index, stream, q.data_ptr(), stride,
          cache, cu_p, len_p, o.data_ptr(), None if lse is None else lse.data_ptr(), B, Hq, total,
          total if max_q is None else max_q, d ** -0.5 if scale is None else scale, window)
    return o, lse


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
    return torch.tensor(list(buf), dtype=_F64), amp.value


def _turns_of(turns, index, d):
    """Rotated values of a head: two for each entry of `turns`."""
    shape = turns.shape
    if turns.dtype is not _F64 or len(shape) != 1 or turns.get_device() != index or \
            not turns.is_contiguous():
        raise ValueError(f"turns must be a contiguous float64 tensor [rot / 2] on cuda:{index}")
    rot = 2 * shape[0]
    if rot > d:
        raise ValueError("turns must have at most d / 2 entries")
    return rot


_Strides = _L * 12


def _strides3(t, shape):
    """Batch, head and token strides (0 where a dimension has one element)."""
    s = t.stride()
    if s[3] != 1 and shape[3] > 1:
        raise ValueError("the last dimension of q, k and the outputs must be contiguous")
    return (s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0, s[2] if shape[2] > 1 else 0)


def _rope_out(x, shape, out, dtype, index):
    if out is None:
        return _empty(shape, device=x.device, dtype=dtype)
    if out.shape != shape or out.dtype is not dtype or out.get_device() != index:
        raise ValueError("an output must have its input's shape, type and device")
    return out


def _rope(q, k, pos, turns, amp, interleaved, q_out, k_out, stream, backward):
    dtype, index, shape = q.dtype, q.get_device(), q.shape
    if dtype is not _BF16 and dtype is not _F16:
        raise ValueError("q must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if len(shape) != 4:
        raise ValueError("q must be a 4-D tensor [B, H, N, d]")
    B, Hq, N, d = shape
    strides = _strides3(q, shape)
    q_out = _rope_out(q, shape, q_out, dtype, index)
    strides += _strides3(q_out, shape)
    Hkv, k_p, k_out_p = 0, None, None
    if k is not None:
        kshape = k.shape
        if len(kshape) != 4 or k.dtype is not dtype or k.get_device() != index or \
                kshape[0] != B or kshape[2] != N or kshape[3] != d:
            raise ValueError("k must be [B, Hkv, N, d] of q's B, N, d, type and device")
        Hkv = kshape[1]
        strides += _strides3(k, kshape)
        k_out = _rope_out(k, kshape, k_out, dtype, index)
        strides += _strides3(k_out, kshape)
        k_p, k_out_p = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    at = pos.shape
    if pos.dtype is not _I32 or pos.get_device() != index or not pos.is_contiguous() or \
            (at != (N,) and at != (B, N)):
        raise ValueError(f"pos must be a contiguous int32 tensor [N] or [B, N] on cuda:{index}")
    rot = _turns_of(turns, index, d)
    _call("attn_rope_f16" if dtype is _F16 else "attn_rope", index, stream, q.data_ptr(),
          q_out.data_ptr(), k_p, k_out_p, _Strides(*strides), pos.data_ptr(),
          N if len(at) == 2 else 0, turns.data_ptr(), B, Hq, Hkv, N, d, rot, amp,
          1 if interleaved else 0, backward)
    return q_out, k_out


def attn_rope(q, k, pos, turns, amp: float = 1.0, interleaved: bool = False, q_out=None,
              k_out=None, stream=None) -> Tuple:
    """Rotary positions of q [B, Hq, N, d] and k [B, Hkv, N, d] (or None), bf16 or fp16.

    Any strides with d innermost; an output may be its input. pos int32 [N] or
    [B, N]; turns and amp from ``attn_rope_turns`` (turns on q's device): the
    first 2 * len(turns) values of each head are rotated. Returns (q_out, k_out).
    """
    return _rope(q, k, pos, turns, amp, interleaved, q_out, k_out, stream, 0)


def attn_rope_bwd(dq, dk, pos, turns, amp: float = 1.0, interleaved: bool = False, dq_in=None,
                  dk_in=None, stream=None) -> Tuple:
    """Gradients of ``attn_rope``'s inputs from those of its outputs (same arguments)."""
    return _rope(dq, dk, pos, turns, amp, interleaved, dq_in, dk_in, stream, 1)


def attn_rope_append(q, k, v, kpages, vpages, table, cu_q, kv_lens, turns, amp: float = 1.0,
                     interleaved: bool = False, pos=None, q_out=None, stream=None):
    """Rotate new tokens' q and k, and put k and v into the paged cache, in one pass.

    q [total, Hq, d], k and v [total, Hkv, d] (rows may be parts of wider ones, as
    one projection gives them); cache arguments as in ``attn_paged``. Positions
    are the tokens' places in the cache unless pos (int32 [total]) is given.
    Returns q_out; the pools are updated in place.
    """
    cache, index, layers, _, B = _cache(kpages, vpages, table)
    if layers:
        raise ValueError("kpages must be one layer's pool [num_pages, Hkv, page_size, d]")
    dtype, d, Hkv = kpages.dtype, cache.d, cache.Hkv
    shape, qs = _packed(q, "q", dtype, index, None, d)
    total, Hq = shape[0], shape[1]
    kshape, ks = _packed(k, "k", dtype, index, Hkv, d)
    vshape, vs = _packed(v, "v", dtype, index, Hkv, d)
    if kshape[0] != total or vshape[0] != total:
        raise ValueError("q, k and v must have the same tokens")
    cu_p = _int32(cu_q, "cu_q", index, (B + 1,))
    len_p = _int32(kv_lens, "kv_lens", index, (B,))
    pos_p = None if pos is None else _int32(pos, "pos", index, (total,))
    if q_out is None:
        q_out, os_ = _empty(shape, device=q.device, dtype=dtype), Hq * d
    else:
        oshape, os_ = _packed(q_out, "q_out", dtype, index, Hq, d)
        if oshape != shape:
            raise ValueError("q_out must have q's shape")
    rot = _turns_of(turns, index, d)
    _call("attn_rope_append_f16" if dtype is _F16 else "attn_rope_append", index, stream,
          q.data_ptr(), qs, q_out.data_ptr(), os_, k.data_ptr(), ks, v.data_ptr(), vs, cache, cu_p,
          len_p, pos_p, turns.data_ptr(), B, Hq, total, rot, amp, 1 if interleaved else 0)
    return q_out


def _next(t, out, name, index, shape):
    """(out or a new tensor like t, its address)."""
    if out is None:
        out = _empty_like(t)
        return out, out.data_ptr()
    return out, _int32(out, name, index, shape)


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
    cache, index, layers, layer_stride, B = _cache(kpages, vpages, table)
    rows, pages = (B,), (cache.num_pages,)
    len_p = _int32(lens, "lens", index, rows)
    ref_p = _int32(refs, "refs", index, pages)
    src_p = _int32(source, "source", index, rows)
    add_p = _int32(add, "add", index, rows)
    table_out, t_p = _next(table, table_out, "table_out", index, table.shape)
    lens_out, l_p = _next(lens, lens_out, "lens_out", index, rows)
    refs_out, r_p = _next(refs, refs_out, "refs_out", index, pages)
    if info is None:
        info = _empty(2, dtype=_I32, device=kpages.device)
    i_p = _int32(info, "info", index, (2,))
    _call("attn_pages_update", index, stream, cache, layers or 1, layer_stride, len_p, ref_p, src_p,
          add_p, t_p, l_p, r_p, i_p, B)
    return table_out, lens_out, refs_out, info


def attn_pages_compact(kpages, vpages, table, lens, refs, table_out=None, refs_out=None, info=None,
                       stream=None) -> Tuple:
    """Move the live pages to the lowest indices, in every layer, with the fewest copies.

    Arguments as in ``attn_pages_update``. Returns (table, refs, info) of the next
    state; info [2]: live pages, moved pages.
    """
    cache, index, layers, layer_stride, B = _cache(kpages, vpages, table)
    pages = (cache.num_pages,)
    len_p = _int32(lens, "lens", index, (B,))
    ref_p = _int32(refs, "refs", index, pages)
    table_out, t_p = _next(table, table_out, "table_out", index, table.shape)
    refs_out, r_p = _next(refs, refs_out, "refs_out", index, pages)
    if info is None:
        info = _empty(2, dtype=_I32, device=kpages.device)
    i_p = _int32(info, "info", index, (2,))
    _call("attn_pages_compact", index, stream, cache, layers or 1, layer_stride, len_p, ref_p, t_p,
          r_p, i_p, B)
    return table_out, refs_out, info
