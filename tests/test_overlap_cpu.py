"""Outputs over inputs or over one another: refused on the host, before any launch.

Held against the sets of bytes that each call reads and writes. Without a GPU a
call that the checks let pass ends at the device query (ATTN_ERR_CUDA), so the
addresses are never followed.
"""
import ctypes
import itertools
import random

import pytest

import exact_tiled_attention_38_b200 as eta
from exact_tiled_attention_38_b200 import build as eta_build
from test_paged_cpu import pages

INVALID = eta.ATTN_ERR_INVALID
A = 1 << 20


@pytest.fixture(scope="module")
def clib():
    import torch

    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no kernel can run")
    eta_build.build()
    return eta.load_library()


def cells(base, n, s, d):
    """16-byte units of pieces of d values at base + i . s."""
    return {base // 16 + sum(i * t for i, t in zip(at, s)) // 8 + u
            for at in itertools.product(*map(range, n)) for u in range(d // 8)}


def twice(base, n, s, d):
    return len(cells(base, n, s, d)) < n[0] * n[1] * n[2] * (d // 8)


def rope(clib, q, qo, k, ko, B, Hq, Hkv, N, d, rot=None):
    s = (ctypes.c_longlong * 12)(*q[1], *qo[1], *k[1], *ko[1])
    return clib.attn_rope(q[0], qo[0], k[0], ko[0], s, 64, 0, 64, B, Hq, Hkv, N, d, d if rot is None else rot, 1.0,
                          0, 0, None)


def test_rope_against_the_sets(clib):
    r = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        B, Hq, Hkv, N, d = r.randint(1, 3), r.randint(1, 4), r.randint(1, 3), r.randint(1, 4), r.choice([8, 16, 24])
        # parts of one buffer [B, N, H, d] or [B, H, N, d], now and then spread or in other buffers
        H = Hq + Hkv + r.randint(0, 3)
        s = r.choice([(N * H * d, d, H * d), (H * N * d, N * d, d), (N * H * d * 2, 2 * d, 2 * H * d)])
        place = lambda: A + 16 * r.choice([0, 0, d // 8 * r.randint(0, H), r.randint(0, 3 * N * H * d // 8),  # noqa: E731
                                           1 << 14, 1 << 15])
        t = [(place(), s) for _ in range(4)]
        if r.random() < 0.4:
            t[1] = t[0]
        if r.random() < 0.4:
            t[3] = t[2]
        sets = [cells(x, (B, h, N), s, d) for (x, s), h in zip(t, (Hq, Hq, Hkv, Hkv))]
        bad = bool((t[1] != t[0] and sets[1] & sets[0]) or (t[3] != t[2] and sets[3] & sets[2]) or
                   sets[1] & sets[2] or sets[3] & sets[0] or sets[1] & sets[3])
        code = rope(clib, *t, B, Hq, Hkv, N, d)
        assert (code == INVALID) == bad, (t, B, Hq, Hkv, N, d)
        seen[bad] += 1
    assert min(seen.values()) > 500


def test_rope_outputs_over_themselves(clib):
    r = random.Random(2)
    far = (A + (1 << 24), (4096, 512, 64))
    bad = 0
    for _ in range(3000):
        B, H, N, d = r.randint(1, 3), r.randint(1, 4), r.randint(1, 4), r.choice([8, 16])
        s = tuple(8 * r.choice([0, 1, 2, 3, 4, 8, 16, 64]) for _ in range(3))
        over = twice(A, (B, H, N), s, d)
        code = rope(clib, far, (A, s), (0, (0, 0, 0)), (0, (0, 0, 0)), B, H, 0, N, d)
        if over:
            assert code == INVALID, (B, H, N, d, s)
        else:  # passes, or its strides do not nest
            by = sorted((t, n) for t, n in zip(s, (B, H, N)) if n > 1)
            nests, extent = True, d
            for t, n in by:
                nests, extent = nests and t >= extent, extent + (n - 1) * t
            assert (code == INVALID) == (not nests), (B, H, N, d, s)
        bad += over
        # an input may have its values in one place (a broadcast one)
        assert rope(clib, (A, s), far, (0, (0, 0, 0)), (0, (0, 0, 0)), B, H, 0, N, d) != INVALID
    assert 300 < bad < 2700


def test_rope_other_strides(clib):
    one, none = (4096, 512, 64), (0, (0, 0, 0))
    # q's memory in another layout; with one head or token the stride does not count
    assert rope(clib, (A, one), (A, (4096, 64, 512)), none, none, 2, 8, 0, 8, 64) == INVALID
    assert rope(clib, (A, one), (A, (4096, 64, 64)), none, none, 2, 1, 0, 8, 64) != INVALID
    assert rope(clib, (A, one), (A, (0, 512, 64)), none, none, 1, 8, 0, 8, 64) != INVALID
    assert rope(clib, (A, (1 << 50, 512, 64)), (A + (1 << 30), one), none, none, 2, 8, 0, 8, 64) == INVALID


def test_append_against_the_sets(clib):
    r = random.Random(3)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        total, Hq, Hkv = r.randint(1, 5), r.randint(1, 3), r.randint(1, 2)
        d, row = 8, (Hq + 2 * Hkv + r.randint(0, 4)) * 8
        place = lambda: A + 16 * r.choice([0, Hq, Hq + Hkv, r.randint(0, 5 * row // 8), 1 << 12])  # noqa: E731
        q, qo, k, v = (place() for _ in range(4))
        if r.random() < 0.4:
            qo = q
        c = lambda x, h: cells(x, (total, 1, 1), (row, 0, 0), h * d)  # noqa: E731
        bad = bool((qo != q and c(qo, Hq) & c(q, Hq)) or c(qo, Hq) & c(k, Hkv) or c(qo, Hq) & c(v, Hkv))
        pool = pages(d=8, Hkv=Hkv, token_stride=8, head_stride=128, page_stride=128 * Hkv)
        code = clib.attn_rope_append(q, row, qo, row, k, row, v, row, pool, 64, 64, None, 64, 2, Hq, total, 8, 1.0,
                                     0, None)
        assert (code == INVALID) == bad, (q, qo, k, v, total, Hq, Hkv, row)
        seen[bad] += 1
    assert min(seen.values()) > 500
    # in place with another stride
    pool = pages(d=8, Hkv=1, token_stride=8, head_stride=128, page_stride=128)
    args = lambda s, t: (A, 64, A, s, 2 * A, 64, 2 * A, 64, pool, 64, 64, None, 64, 2, 4, t, 8, 1.0, 0, None)  # noqa: E731
    assert clib.attn_rope_append(*args(32, 3)) == INVALID
    assert clib.attn_rope_append(*args(32, 1)) != INVALID  # one token: no stride counts


def test_paged_against_the_sets(clib):
    r = random.Random(4)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        total, Hq = r.randint(1, 5), r.choice([2, 4])
        row = (Hq + r.choice([0, 4, 40])) * 8
        q, o = (A + 16 * r.randint(0, 60) for _ in range(2))
        lse = r.choice([None, A + 4 * r.randint(0, 600), 8 * A])
        c = cells(q, (total, 1, 1), (row, 0, 0), Hq * 8)
        at_o = cells(o, (1, 1, 1), (0, 0, 0), total * Hq * 8)
        qb = {16 * x + u for x in c for u in range(16)}
        ob = {16 * x + u for x in at_o for u in range(16)}
        lb = set(range(lse, lse + total * Hq * 4)) if lse else set()
        bad = bool(ob & qb or lb & qb or lb & ob)
        pool = pages(d=8, Hkv=2, token_stride=8, head_stride=128, page_stride=256)
        code = clib.attn_paged(q, row, pool, 64, 64, o, lse, 2, Hq, total, 3, 0.1, 0, None)
        assert (code == INVALID) == bad, (q, o, lse, total, Hq, row)
        seen[bad] += 1
    assert min(seen.values()) > 500


def test_page_operations(clib):
    B, P, W = 3, 10, 4
    size = dict(table=4 * B * W, lens=4 * B, refs=4 * P, source=4 * B, add=4 * B, table_out=4 * B * W, lens_out=4 * B,
                refs_out=4 * P, info=8)
    names = list(size)

    def call(at):
        c = pages(table=at["table"])
        u = clib.attn_pages_update(c, 1, 0, *(at[n] for n in names[1:]), B, None)
        m = clib.attn_pages_compact(c, 1, 0, at["lens"], at["refs"], at["table_out"], at["refs_out"], at["info"], B,
                                    None)
        return u, m

    apart = {n: A + 1024 * i for i, n in enumerate(names)}
    assert INVALID not in call(apart)
    only_update = {"source", "add", "lens_out"}
    for x, y in itertools.permutations(names, 2):
        for by in (0, 4, size[y] - 4, size[y], -size[x], 4 - size[x]):
            at = dict(apart)
            at[x] = at[y] + by
            bad = -size[x] < by < size[y] and (x in names[5:] or y in names[5:])
            u, m = call(at)
            assert (u == INVALID) == bad, (x, y, by)
            assert (m == INVALID) == (bad and not {x, y} & only_update), (x, y, by)
