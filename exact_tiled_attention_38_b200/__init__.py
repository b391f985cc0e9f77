"""Python binding for the exact tiled attention library (``include/attn.h``).

Argument marshalling only: every function checks shapes and dtypes of torch
tensors, then calls the C entry point of the same name with raw device
pointers and the current CUDA stream. All arithmetic runs in the CUDA kernels
of ``libattn.so``; there is no fallback path. If the library is missing or
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libattn.so")

ATTN_OK = 0
ATTN_ERR_INVALID = -1
ATTN_ERR_UNSUPPORTED = -2
ATTN_ERR_CUDA = -3
ATTN_ERR_TIMEOUT = -4
ATTN_ERR_SCRATCH = -5
ATTN_ERR_PAGES = -6

# name -> (restype, argtypes); mirrors include/attn.h
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_L = ctypes.c_longlong
_D = ctypes.c_double


class _Pages(ctypes.Structure):
    """``attn_pages`` of include/attn.h."""
    _fields_ = [("k", _P), ("v", _P), ("table", _P), ("page_stride", _L), ("head_stride", _L),
                ("token_stride", _L), ("num_pages", _I), ("page_size", _I), ("table_width", _I),
                ("Hkv", _I), ("d", _I)]


_PP = ctypes.POINTER(_Pages)
_PAGED = [_P, _L, _PP, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]
_ROPE = [_P, _P, _P, _P, ctypes.POINTER(_L), _P, _L, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]
_APPEND = [_P, _L, _P, _L, _P, _L, _P, _L, _PP, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]
SIGNATURES = {
    "attn_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_fwd_f16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P]),
    "attn_decode_f16": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P]),
    "attn_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P]),
    "attn_decode_num_splits": (_I, [_I, _I, _I, _I]),
    "attn_strerror": (ctypes.c_char_p, [_I]),
    "attn_get_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_uint)]),
    "attn_fwd_stall_test": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I,
                                 ctypes.c_uint, _P]),
    "attn_fwd_window": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_fwd_window_f16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_decode_window": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "attn_decode_window_f16": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _F, _I, _P]),
    "attn_last_cuda_error": (_I, []),
    "attn_merge": (_I, [_P, _P, _P, _P, _P, ctypes.c_longlong, _I, _P]),
    "attn_merge_f16": (_I, [_P, _P, _P, _P, _P, ctypes.c_longlong, _I, _P]),
    "attn_fwd_partial": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_fwd_partial_f16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "attn_merge_partial": (_I, [_P, _P, _P, _P, _P, ctypes.c_longlong, _I, _P]),
    "attn_merge_partial_f16": (_I, [_P, _P, _P, _P, _P, ctypes.c_longlong, _I, _P]),
    "attn_paged": (_I, _PAGED),
    "attn_paged_f16": (_I, _PAGED),
    "attn_rope": (_I, _ROPE),
    "attn_rope_f16": (_I, _ROPE),
    "attn_rope_append": (_I, _APPEND),
    "attn_rope_append_f16": (_I, _APPEND),
    "attn_rope_turns": (_I, [ctypes.POINTER(_D), ctypes.POINTER(_F), _I, _D, _I, _D, _D, _D, _D]),
    "attn_pages_update": (_I, [_PP, _I, _L, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P]),
    "attn_pages_compact": (_I, [_PP, _I, _L, _P, _P, _P, _P, _P, _I, _P]),
}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        self.cuda_error = load_library().attn_last_cuda_error() if code == ATTN_ERR_CUDA else 0
        extra = f", cudaError {self.cuda_error}" if self.cuda_error else ""
        super().__init__(f"{where}: {strerror(code)} (code {code}{extra})")


def load_library(path: str = LIB_PATH):
    """Load ``libattn.so`` (once). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run `python -m exact_tiled_attention_38_b200.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load_library().attn_strerror(int(code)).decode()


def _stream_handle(stream) -> Optional[int]:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, int):
        return stream or None
    return stream.cuda_stream or None


def _check(code: int, where: str):
    if code != ATTN_OK:
        raise AttnError(code, where)


def _dev(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on_device(*tensors):
    """The library works on the current CUDA device: every tensor of a call must
    live on one device, which is made current for the call (and whose current
    stream is used when none is given)."""
    import torch

    devs = {t.device for t in tensors if t is not None}
    if len(devs) != 1:
        raise ValueError(f"all tensors of a call must be on one CUDA device, got {sorted(map(str, devs))}")
    return torch.cuda.device(next(iter(devs)))


def _fwd(fname, dtype, q, k, v, o, lse, scale, causal, stream, want_lse, window=None,
         out_dtype=None):
    import torch

    out_dtype = out_dtype or dtype
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dev(t, n)
        if t.dtype != dtype or t.dim() != 4:
            raise ValueError(f"{n} must be a 4-D {dtype} tensor [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    Bk, Hkv, Nk, dk = k.shape
    if Bk != B or dk != d or tuple(v.shape) != tuple(k.shape):
        raise ValueError("q/k/v shapes disagree")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty(q.shape, device=q.device, dtype=out_dtype)
    _dev(o, "o")
    if o.dtype != out_dtype or tuple(o.shape) != tuple(q.shape):
        raise ValueError(f"o must be a {out_dtype} tensor of q's shape")
    if lse is None and want_lse:
        lse = torch.empty((B, Hq, Nq), device=q.device, dtype=torch.float32)
    if lse is not None:
        _dev(lse, "lse")
        if lse.dtype != torch.float32 or tuple(lse.shape) != (B, Hq, Nq):
            raise ValueError("lse must be float32 [B, Hq, Nq]")
    fn = getattr(load_library(), fname)
    with _on_device(q, k, v, o, lse):
        code = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                  lse.data_ptr() if lse is not None else None, B, Hq, Hkv, Nq, Nk, d,
                  float(scale), *((int(window),) if window is not None else (1 if causal else 0,)),
                  _stream_handle(stream))
    _check(code, fname)
    return o, lse


def attn_fwd(q, k, v, o=None, lse=None, scale: Optional[float] = None, causal: bool = False,
             stream=None, want_lse: bool = True) -> Tuple:
    """Prefill attention, bf16. q [B,Hq,Nq,d], k/v [B,Hkv,Nk,d] -> (o, lse)."""
    import torch

    return _fwd("attn_fwd", torch.bfloat16, q, k, v, o, lse, scale, causal, stream, want_lse)


def attn_fwd_f16(q, k, v, o=None, lse=None, scale: Optional[float] = None,
                 causal: bool = False, stream=None, want_lse: bool = True) -> Tuple:
    """Prefill attention, fp16."""
    import torch

    return _fwd("attn_fwd_f16", torch.float16, q, k, v, o, lse, scale, causal, stream,
                want_lse)


def attn_fwd_partial(q, k, v, o=None, lse=None, scale: Optional[float] = None,
                     causal: bool = False, stream=None, want_lse: bool = True) -> Tuple:
    """Prefill attention with O kept in float32 (unrounded), for results that
    are merged further (``attn_merge`` with a float32 ``o_part``). q, k, v bf16
    or fp16; returns (o float32 [B,Hq,Nq,d], lse)."""
    import torch

    if q.dtype == torch.float16:
        name, dt = "attn_fwd_partial_f16", torch.float16
    else:
        name, dt = "attn_fwd_partial", torch.bfloat16
    return _fwd(name, dt, q, k, v, o, lse, scale, causal, stream, want_lse,
                out_dtype=torch.float32)


def _decode(fname, dtype, q, kcache, vcache, seqlens, Hkv, o, lse, scale, stream, want_lse,
            window=None):
    import torch

    for t, n in ((q, "q"), (kcache, "kcache"), (vcache, "vcache"), (seqlens, "seqlens")):
        _dev(t, n)
    if q.dtype != dtype or q.dim() != 3:
        raise ValueError(f"q must be a 3-D {dtype} tensor [B, Hq, d]")
    if kcache.dtype != dtype or vcache.dtype != dtype:
        raise ValueError(f"caches must be {dtype}")
    if seqlens.dtype != torch.int32:
        raise ValueError("seqlens must be int32")
    B, Hq, d = q.shape
    if seqlens.numel() != B:
        raise ValueError("seqlens must have B entries")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if o is None:
        o = torch.empty_like(q)
    _dev(o, "o")
    if lse is None and want_lse:
        lse = torch.empty((B, Hq), device=q.device, dtype=torch.float32)
    fn = getattr(load_library(), fname)
    with _on_device(q, kcache, vcache, seqlens, o, lse):
        code = fn(q.data_ptr(), kcache.data_ptr(), vcache.data_ptr(), seqlens.data_ptr(),
                  o.data_ptr(), lse.data_ptr() if lse is not None else None, B, Hq, Hkv, d,
                  float(scale), *((int(window),) if window is not None else ()),
                  _stream_handle(stream))
    _check(code, fname)
    return o, lse


def attn_fwd_window(q, k, v, window: int, o=None, lse=None, scale: Optional[float] = None,
                    stream=None, want_lse: bool = True) -> Tuple:
    """Causal prefill with a sliding window of `window` keys, bf16 (fp16 if q is fp16)."""
    import torch

    name, dt = (("attn_fwd_window_f16", torch.float16) if q.dtype == torch.float16
                else ("attn_fwd_window", torch.bfloat16))
    return _fwd(name, dt, q, k, v, o, lse, scale, True, stream, want_lse, window=window)


def attn_decode_window(q, kcache, vcache, seqlens, Hkv: int, window: int, o=None, lse=None,
                       scale: Optional[float] = None, stream=None, want_lse: bool = True):
    """Decode reading the last `window` cached tokens, bf16 (fp16 if q is fp16)."""
    import torch

    name, dt = (("attn_decode_window_f16", torch.float16) if q.dtype == torch.float16
                else ("attn_decode_window", torch.bfloat16))
    return _decode(name, dt, q, kcache, vcache, seqlens, Hkv, o, lse, scale, stream, want_lse,
                   window=window)


def attn_decode(q, kcache, vcache, seqlens, Hkv: int, o=None, lse=None,
                scale: Optional[float] = None, stream=None, want_lse: bool = True):
    """One-token decode over a packed ragged cache, bf16. Returns (o [B,Hq,d], lse [B,Hq])."""
    import torch

    return _decode("attn_decode", torch.bfloat16, q, kcache, vcache, seqlens, Hkv, o, lse,
                   scale, stream, want_lse)


def attn_decode_f16(q, kcache, vcache, seqlens, Hkv: int, o=None, lse=None,
                    scale: Optional[float] = None, stream=None, want_lse: bool = True):
    """One-token decode, fp16."""
    import torch

    return _decode("attn_decode_f16", torch.float16, q, kcache, vcache, seqlens, Hkv, o, lse,
                   scale, stream, want_lse)


def attn_decode_noalloc(q, kcache, vcache, seqlens, Hkv: int, o=None, lse=None,
                        scale: Optional[float] = None, stream=None, want_lse: bool = True):
    """bf16 decode whose scratch is the library's fixed device array.

    For callers that cannot allocate device memory where decode runs. The
    library allocates nothing here; pass preallocated ``o`` / ``lse`` to keep
    this wrapper from allocating them either. Calls that may overlap on the GPU
    share the scratch and must be ordered (one stream, or events).
    """
    import torch

    return _decode("attn_decode_noalloc", torch.bfloat16, q, kcache, vcache, seqlens, Hkv, o,
                   lse, scale, stream, want_lse)


def attn_merge(o_acc, lse_acc, o_part, lse_part, o_out=None, stream=None) -> None:
    """Fold a partial result (o_part, lse_part) into the fp32 accumulator in place.

    o_acc float32 [..., d] and lse_acc float32 [...] (same leading shape as
    o_part / lse_part); o_part bf16, fp16 or float32 (an unrounded partial from
    ``attn_fwd_partial``); o_out (optional, o_part's shape; bf16 or fp16, o_part's
    dtype unless o_part is float32) also receives the merged O rounded. A row
    with lse_acc = -inf is empty (o_acc not read). Runs ``attn_merge`` /
    ``attn_merge_f16``, or ``attn_merge_partial`` / ``attn_merge_partial_f16``.
    """
    import torch

    for t, n in ((o_acc, "o_acc"), (lse_acc, "lse_acc"), (o_part, "o_part"),
                 (lse_part, "lse_part")):
        _dev(t, n)
    if o_part.dtype not in (torch.bfloat16, torch.float16, torch.float32):
        raise ValueError("o_part must be bf16, fp16 or float32")
    if o_acc.dtype != torch.float32 or lse_acc.dtype != torch.float32 or \
            lse_part.dtype != torch.float32:
        raise ValueError("o_acc, lse_acc and lse_part must be float32")
    d = o_part.shape[-1]
    if tuple(o_acc.shape) != tuple(o_part.shape) or \
            tuple(lse_acc.shape) != tuple(o_part.shape[:-1]) or \
            tuple(lse_part.shape) != tuple(o_part.shape[:-1]):
        raise ValueError("o_acc, lse_acc, o_part and lse_part shapes disagree")
    if o_out is not None:
        _dev(o_out, "o_out")
        if tuple(o_out.shape) != tuple(o_part.shape) or (
                o_out.dtype != o_part.dtype if o_part.dtype != torch.float32
                else o_out.dtype not in (torch.bfloat16, torch.float16)):
            raise ValueError("o_out must match o_part's shape (and dtype, or bf16 / fp16 "
                             "for a float32 o_part)")
    if o_part.dtype == torch.float32:
        f16 = o_out is not None and o_out.dtype == torch.float16
        name = "attn_merge_partial_f16" if f16 else "attn_merge_partial"
    else:
        name = "attn_merge_f16" if o_part.dtype == torch.float16 else "attn_merge"
    rows = o_part.numel() // d if d else 0
    with _on_device(o_acc, lse_acc, o_part, lse_part, o_out):
        code = getattr(load_library(), name)(
            o_acc.data_ptr(), lse_acc.data_ptr(), o_part.data_ptr(), lse_part.data_ptr(),
            o_out.data_ptr() if o_out is not None else None, rows, d, _stream_handle(stream))
    _check(code, name)


def attn_decode_num_splits(B: int, Hq: int, Hkv: int, d: int) -> int:
    r = load_library().attn_decode_num_splits(B, Hq, Hkv, d)
    if r < 0:
        raise AttnError(r, "attn_decode_num_splits")
    return r


def attn_get_device_status(stream=None) -> Tuple[int, int]:
    """(status code, raw site code) after synchronising the stream; clears the word."""
    raw = ctypes.c_uint(0)
    code = load_library().attn_get_device_status(_stream_handle(stream), ctypes.byref(raw))
    return code, raw.value


# ---------------------------------------------------------------- paged cache
# A decode step makes these calls every few microseconds, so their checks are
# kept short: one pass over the arguments, no context switch when the tensors'
# device is the current one.

def _call(fn, device, stream, *args):
    """Run entry point `fn` with `args` and a stream on `device`."""
    import torch

    f = getattr(_lib or load_library(), fn)
    if device.index == torch.cuda.current_device():
        code = f(*args, _raw_stream(device) if stream is None else _stream_handle(stream))
    else:
        with torch.cuda.device(device):
            code = f(*args, _raw_stream(device) if stream is None else _stream_handle(stream))
    if code != ATTN_OK:
        raise AttnError(code, fn)


def _raw_stream(device):
    import torch

    return torch.cuda.current_stream(device).cuda_stream or None


def _int32(t, name, device, shape):
    import torch

    if t.dtype != torch.int32 or t.device != device or tuple(t.shape) != shape or \
            not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {shape} on {device}")


def _cache(kpages, vpages, table):
    """(_Pages, layers, layer_stride) of pools [num_pages, Hkv, page_size, d], or
    [layers, num_pages, Hkv, page_size, d], in any strides with d innermost."""
    import torch

    dtype, device = kpages.dtype, kpages.device
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise ValueError("kpages and vpages must be bf16 or fp16")
    if not kpages.is_cuda:
        raise ValueError("kpages must be a CUDA tensor")
    shape, strides = kpages.shape, kpages.stride()
    if vpages.dtype != dtype or vpages.device != device or vpages.shape != shape or \
            vpages.stride() != strides:
        raise ValueError("vpages must have kpages' type, device, shape and strides")
    layers, layer_stride = 1, 0
    if len(shape) == 5:
        layers, layer_stride = shape[0], strides[0]
        shape, strides = shape[1:], strides[1:]
    if len(shape) != 4 or strides[3] != 1:
        raise ValueError("kpages must be [num_pages, Hkv, page_size, d] (or with layers in front), "
                         "d innermost")
    if table.dtype != torch.int32 or table.device != device or table.dim() != 2 or \
            not table.is_contiguous():
        raise ValueError(f"table must be a contiguous int32 tensor [B, width] on {device}")
    P, Hkv, page, d = shape
    # A dimension of one element has no stride that matters: give it the packed one.
    token = strides[2] if page > 1 else d
    head = strides[1] if Hkv > 1 else page * d
    stride = strides[0] if P > 1 else max(Hkv * page * d, 8)
    return (_Pages(kpages.data_ptr(), vpages.data_ptr(), table.data_ptr(), stride, head, token, P,
                   page, table.shape[1], Hkv, d), layers, layer_stride)


def _packed(t, name, like, heads, d):
    """Token stride of a packed tensor [total, heads, d] whose rows may be parts of wider ones."""
    if t.dtype != like.dtype or t.device != like.device or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D {like.dtype} tensor [tokens, heads, d] on {like.device}")
    if t.shape[2] != d or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must have {heads if heads is not None else 'its'} heads of {d}")
    s = t.stride()
    if (s[2] != 1 and d > 1) or (s[1] != d and t.shape[1] > 1):
        raise ValueError(f"the heads of a token of {name} must be contiguous")
    return s[0] if t.shape[0] > 1 else t.shape[1] * d


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
    import torch

    cache, layers, _ = _cache(kpages, vpages, table)
    if layers != 1 or kpages.dim() != 4:
        raise ValueError("kpages must be one layer's pool [num_pages, Hkv, page_size, d]")
    device, B = kpages.device, table.shape[0]
    stride = _packed(q, "q", kpages, None, cache.d)
    total, Hq, d = q.shape
    _int32(cu_q, "cu_q", device, (B + 1,))
    _int32(kv_lens, "kv_lens", device, (B,))
    if o is None:
        o = torch.empty((total, Hq, d), device=device, dtype=q.dtype)
    elif o.dtype != q.dtype or o.device != device or o.shape != q.shape or not o.is_contiguous():
        raise ValueError("o must be a contiguous tensor of q's shape, type and device")
    if lse is None:
        if want_lse:
            lse = torch.empty((total, Hq), device=device, dtype=torch.float32)
    elif lse.dtype != torch.float32 or lse.device != device or \
            tuple(lse.shape) != (total, Hq) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 tensor [total, Hq] on q's device")
    _call("attn_paged_f16" if q.dtype == torch.float16 else "attn_paged", device, stream,
          q.data_ptr(), stride, cache, cu_q.data_ptr(), kv_lens.data_ptr(), o.data_ptr(),
          lse.data_ptr() if lse is not None else None, B, Hq, total,
          total if max_q is None else int(max_q),
          1.0 / math.sqrt(d) if scale is None else float(scale), int(window))
    return o, lse


def attn_rope_turns(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                    low: float = 1.0, high: Optional[float] = None, original: float = 4096.0):
    """Turns per position of each rotary pair (float64, on the CPU) and the amplitude.

    scaling: "none", "linear", "base", "parts" (high defaults to 32) or "bands"
    (high defaults to 4); see ``attn_rope_turns`` in include/attn.h.
    """
    import torch

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


def _turns_of(turns, device, d):
    import torch

    if turns.dtype != torch.float64 or turns.device != device or turns.dim() != 1 or \
            not turns.is_contiguous():
        raise ValueError(f"turns must be a contiguous float64 tensor [rot / 2] on {device}")
    rot = 2 * turns.shape[0]
    if rot > d:
        raise ValueError("turns must have at most d / 2 entries")
    return rot


def _rope(q, k, pos, turns, amp, interleaved, q_out, k_out, stream, backward):
    import torch

    dtype, device = q.dtype, q.device
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise ValueError("q must be bf16 or fp16")
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    if q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [B, H, N, d]")
    B, Hq, N, d = q.shape
    Hkv = 0
    if k is not None:
        if k.dim() != 4 or k.dtype != dtype or k.device != device or \
                (k.shape[0], k.shape[2], k.shape[3]) != (B, N, d):
            raise ValueError("k must be [B, Hkv, N, d] of q's B, N, d, type and device")
        Hkv = k.shape[1]
    elif k_out is not None:
        raise ValueError("k_out without k")
    if q_out is None:
        q_out = torch.empty((B, Hq, N, d), device=device, dtype=dtype)
    if k is not None and k_out is None:
        k_out = torch.empty((B, Hkv, N, d), device=device, dtype=dtype)
    strides = (_L * 12)()
    at = 0
    for t, like in ((q, q), (q_out, q), (k, k), (k_out, k)):
        if t is not None:
            if t.shape != like.shape or t.dtype != dtype or t.device != device:
                raise ValueError("an output must have its input's shape, type and device")
            s, n = t.stride(), t.shape
            if s[3] != 1 and d > 1:
                raise ValueError("the last dimension of q, k and the outputs must be contiguous")
            # A dimension of one element has no stride that matters.
            strides[at] = s[0] if n[0] > 1 else 0
            strides[at + 1] = s[1] if n[1] > 1 else 0
            strides[at + 2] = s[2] if n[2] > 1 else 0
        at += 3
    if pos.dtype != torch.int32 or pos.device != device or not pos.is_contiguous() or \
            tuple(pos.shape) not in ((N,), (B, N)):
        raise ValueError(f"pos must be a contiguous int32 tensor [N] or [B, N] on {device}")
    rot = _turns_of(turns, device, d)
    _call("attn_rope_f16" if dtype == torch.float16 else "attn_rope", device, stream,
          q.data_ptr(), q_out.data_ptr(), k.data_ptr() if k is not None else None,
          k_out.data_ptr() if k is not None else None, strides, pos.data_ptr(),
          N if pos.dim() == 2 else 0, turns.data_ptr(), B, Hq, Hkv, N, d, rot, float(amp),
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
    import torch

    cache, layers, _ = _cache(kpages, vpages, table)
    if layers != 1 or kpages.dim() != 4:
        raise ValueError("kpages must be one layer's pool [num_pages, Hkv, page_size, d]")
    device, B, d = kpages.device, table.shape[0], cache.d
    total, Hq = q.shape[0], q.shape[1] if q.dim() == 3 else 0
    qs = _packed(q, "q", kpages, None, d)
    ks = _packed(k, "k", kpages, cache.Hkv, d)
    vs = _packed(v, "v", kpages, cache.Hkv, d)
    if k.shape[0] != total or v.shape[0] != total:
        raise ValueError("q, k and v must have the same tokens")
    _int32(cu_q, "cu_q", device, (B + 1,))
    _int32(kv_lens, "kv_lens", device, (B,))
    if pos is not None:
        _int32(pos, "pos", device, (total,))
    if q_out is None:
        q_out = torch.empty((total, Hq, d), device=device, dtype=q.dtype)
    elif q_out.shape != q.shape:
        raise ValueError("q_out must have q's shape")
    os_ = _packed(q_out, "q_out", kpages, Hq, d)
    rot = _turns_of(turns, device, d)
    _call("attn_rope_append_f16" if q.dtype == torch.float16 else "attn_rope_append", device,
          stream, q.data_ptr(), qs, q_out.data_ptr(), os_, k.data_ptr(), ks, v.data_ptr(), vs,
          cache, cu_q.data_ptr(), kv_lens.data_ptr(), pos.data_ptr() if pos is not None else None,
          turns.data_ptr(), B, Hq, total, rot, float(amp), 1 if interleaved else 0)
    return q_out


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
    import torch

    cache, layers, layer_stride = _cache(kpages, vpages, table)
    device, B = kpages.device, table.shape[0]
    for t, n, size in ((lens, "lens", B), (refs, "refs", cache.num_pages),
                       (source, "source", B), (add, "add", B)):
        _int32(t, n, device, (size,))
    if table_out is None:
        table_out = torch.empty_like(table)
    if lens_out is None:
        lens_out = torch.empty_like(lens)
    if refs_out is None:
        refs_out = torch.empty_like(refs)
    if info is None:
        info = torch.empty(2, dtype=torch.int32, device=device)
    for t, n, shape in ((table_out, "table_out", tuple(table.shape)), (lens_out, "lens_out", (B,)),
                        (refs_out, "refs_out", (cache.num_pages,)), (info, "info", (2,))):
        _int32(t, n, device, shape)
    _call("attn_pages_update", device, stream, cache, layers, layer_stride, lens.data_ptr(),
          refs.data_ptr(), source.data_ptr(), add.data_ptr(), table_out.data_ptr(),
          lens_out.data_ptr(), refs_out.data_ptr(), info.data_ptr(), B)
    return table_out, lens_out, refs_out, info


def attn_pages_compact(kpages, vpages, table, lens, refs, table_out=None, refs_out=None, info=None,
                       stream=None) -> Tuple:
    """Move the live pages to the lowest indices, in every layer, with the fewest copies.

    Arguments as in ``attn_pages_update``. Returns (table, refs, info) of the next
    state; info [2]: live pages, moved pages.
    """
    import torch

    cache, layers, layer_stride = _cache(kpages, vpages, table)
    device, B = kpages.device, table.shape[0]
    _int32(lens, "lens", device, (B,))
    _int32(refs, "refs", device, (cache.num_pages,))
    if table_out is None:
        table_out = torch.empty_like(table)
    if refs_out is None:
        refs_out = torch.empty_like(refs)
    if info is None:
        info = torch.empty(2, dtype=torch.int32, device=device)
    for t, n, shape in ((table_out, "table_out", tuple(table.shape)),
                        (refs_out, "refs_out", (cache.num_pages,)), (info, "info", (2,))):
        _int32(t, n, device, shape)
    _call("attn_pages_compact", device, stream, cache, layers, layer_stride, lens.data_ptr(),
          refs.data_ptr(), table_out.data_ptr(), refs_out.data_ptr(), info.data_ptr(), B)
    return table_out, refs_out, info
