"""fp64 CPU oracle of the paged-cache operators (test infrastructure only).

Plain definitions in numpy float64, one sequence, one row and one page at a
time. Nothing is shared with the CUDA library.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _f64, attention_ref

__all__ = ["gather_cache", "paged_attention_ref", "paged_error_bound", "rope_ref", "append_ref",
           "update_ref", "compact_ref"]


def gather_cache(pool, row, length) -> np.ndarray:
    """[Hkv, length, d] of one sequence: position t is row t % page of page row[t // page]."""
    pool = np.asarray(pool)
    page = pool.shape[2]
    out = np.zeros((pool.shape[1], length, pool.shape[3]), dtype=pool.dtype)
    for t in range(length):
        out[:, t] = pool[int(row[t // page]), :, t % page]
    return out


def paged_attention_ref(q, kpool, vpool, table, cu_q, lens, scale, window=0):
    """(o [total, Hq, d], lse [total, Hq]); rows outside every sequence are NaN."""
    q, kpool, vpool = _f64(q), _f64(kpool), _f64(vpool)
    total, Hq, d = q.shape
    o = np.full((total, Hq, d), np.nan)
    lse = np.full((total, Hq), np.nan)
    for b in range(len(lens)):
        a, e, L = int(cu_q[b]), int(cu_q[b + 1]), int(lens[b])
        if e == a:
            continue
        k = gather_cache(kpool, table[b], L)[None]
        v = gather_cache(vpool, table[b], L)[None]
        if L == 0:
            o[a:e], lse[a:e] = 0.0, -np.inf
            continue
        ob, lb = attention_ref(q[a:e].transpose(1, 0, 2)[None], k, v, scale, True, window=window)
        o[a:e], lse[a:e] = ob[0].transpose(1, 0, 2), lb[0].T
    return o, lse


def paged_error_bound(q, kpool, vpool, table, cu_q, lens, scale, window, half_step, least):
    """How far a kernel may be off in o (elementwise) and in lse (per row).

    half_step: relative rounding of the 16-bit type (2^-8 bf16, 2^-11 fp16);
    least: its smallest step (the subnormals'). The kernel rounds each
    probability once (relative half_step, or half the smallest step) before the
    value product and the result once; its scores are 32-bit sums of d products,
    off by at most (d + 8) 2^-24 sum |q_c k_c| scale, which is the relative error
    of a probability, as are the 2^-22 of the exponential; sums of n terms add
    n 2^-24. The weights are normalised, so such errors enter o by
    sum p_j |v_j|, and twice (numerator and denominator).
    """
    q, kpool, vpool = _f64(q), _f64(kpool), _f64(vpool)
    d = q.shape[2]
    o, _ = paged_attention_ref(q, kpool, np.abs(vpool), table, cu_q, lens, scale, window)
    eps = np.zeros(q.shape[:2])
    top = np.zeros(q.shape[0])
    G = q.shape[1] // kpool.shape[1]
    for b in range(len(lens)):
        a, e, L = int(cu_q[b]), int(cu_q[b + 1]), int(lens[b])
        if e == a or L == 0:
            continue
        k = np.abs(gather_cache(kpool, table[b], L)).max(1)  # [Hkv, d]: an upper bound per column
        eps[a:e] = (np.abs(q[a:e]) * np.repeat(k, G, 0)[None]).sum(-1) * scale * (d + 8) * 2.0 ** -24
        eps[a:e] += 2.0 ** -21 + L * 2.0 ** -24
        top[a:e] = np.abs(gather_cache(vpool, table[b], L)).max() * L
    bound_o = o * (2 * half_step + 2 * eps[..., None]) * (1 + 2.0 ** -6) + \
        (top * least / 2 + least)[:, None, None]
    return bound_o, eps * 1.01 + 2.0 ** -18


def rope_ref(x, pos, turns, amp, interleaved, backward=False):
    """x [..., N, d] turned by pos [N] (or broadcastable to x's leading shape + [N])."""
    y = _f64(x).copy()
    turns = np.asarray(turns, dtype=np.float64)
    h = turns.size
    a = 2 * math.pi * np.remainder(np.asarray(pos, dtype=np.float64)[..., None] * turns, 1.0)
    if backward:
        a = -a
    c, s = np.cos(a) * amp, np.sin(a) * amp
    xa, xb = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else \
        (slice(0, h), slice(h, 2 * h))
    u, v = y[..., xa].copy(), y[..., xb].copy()
    y[..., xa], y[..., xb] = u * c - v * s, v * c + u * s
    return y


def append_ref(q, k, v, kpool, vpool, table, cu_q, lens, turns, amp, interleaved, pos=None):
    """(q_out, kpool, vpool) in float64 after the append; q rows of no sequence are NaN."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    kp, vp = _f64(kpool).copy(), _f64(vpool).copy()
    out = np.full(q.shape, np.nan)
    page = kp.shape[2]
    for b in range(len(lens)):
        a, e, L = int(cu_q[b]), int(cu_q[b + 1]), int(lens[b])
        for n in range(a, e):
            at = L - (e - n)
            angle = at if pos is None else int(pos[n])
            out[n] = rope_ref(q[n], np.full(q.shape[1], angle), turns, amp, interleaved)
            if at < 0:
                continue
            p, r = int(table[b][at // page]), at % page
            kp[p, :, r] = rope_ref(k[n], np.full(k.shape[1], angle), turns, amp, interleaved)
            vp[p, :, r] = v[n]
    return out, kp, vp


def update_ref(table, lens, refs, source, add, page):
    """(table, lens, refs, info, copies) of the next state; copies: (from, to) pages."""
    table, lens = [list(map(int, r)) for r in table], list(map(int, lens))
    count = list(map(int, refs))
    source, add = list(map(int, source)), [max(0, int(a)) for a in add]
    width, B = len(table[0]) if table else 0, len(lens)
    up = lambda n: -(-n // page)  # noqa: E731
    for b in range(B):
        for p in table[b][:up(lens[b])]:
            if p >= 0:  # (-1: given up)
                count[p] -= 1
    keeper = {}
    for b, s in enumerate(source):
        if s >= 0 and (s == b or s not in keeper):
            keeper[s] = b
    length = [lens[s] if s >= 0 else 0 for s in source]
    longer = [length[b] + add[b] for b in range(B)]
    kept = [up(length[b]) if s >= 0 and keeper[s] == b else length[b] // page
            for b, s in enumerate(source)]
    for b, s in enumerate(source):
        for p in (table[s][:kept[b]] if s >= 0 else []):
            if p >= 0:
                count[p] += 1
    free = [p for p, c in enumerate(count) if c <= 0]
    long_rows = sum(up(n) > width for n in longer)
    need = sum(up(longer[b]) - kept[b] for b in range(B) if up(longer[b]) <= width)
    info = [max(0, need - len(free)), long_rows]
    if info != [0, 0]:
        return table, lens, list(map(int, refs)), info, []
    rows, copies = [], []
    for b, s in enumerate(source):
        new = [free.pop(0) for _ in range(up(longer[b]) - kept[b])]
        if s >= 0 and kept[b] < up(length[b]):
            copies.append((table[s][kept[b]], new[0]))
        for p in new:
            count[p] = 1
        row = (table[s][:kept[b]] if s >= 0 else []) + new
        rows.append(row + [-1] * (width - len(row)))
    return rows, longer, count, info, copies


def compact_ref(table, lens, refs, page):
    """(table, refs, info, moves) of the next state; moves: (from, to) pages."""
    refs = list(map(int, refs))
    n = sum(r > 0 for r in refs)
    of = [p for p in range(n, len(refs)) if refs[p] > 0]
    to = [p for p in range(n) if refs[p] <= 0]
    count = refs[:n] + [0] * (len(refs) - n)
    for a, b in zip(of, to):
        count[b] = refs[a]
    where = dict(zip(of, to))
    rows = [[where.get(int(p), int(p)) if j < -(-int(l) // page) else -1 for j, p in enumerate(r)]
            for r, l in zip(table, lens)]
    return rows, count, [n, len(of)], list(zip(of, to))
