"""Paged-cache operators without a GPU: host refusals, frequency tables, and the
oracle held against the contiguous one and against brute force."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_38_b200 as eta
import oracle
from exact_tiled_attention_38_b200 import build as eta_build
from oracle import paged as ref
from paged_cases import cu, make_cache, randn


@pytest.fixture(scope="module")
def clib():
    eta_build.build()
    return eta.load_library()


A = 0x10000  # an aligned address that is never followed


def pages(**kw):
    a = dict(k=A, v=A, table=A, page_stride=8 * 16 * 128, head_stride=16 * 128, token_stride=128,
             num_pages=10, page_size=16, table_width=4, Hkv=8, d=128)
    a.update(kw)
    return eta._Pages(**a)


INVALID, UNSUPPORTED = eta.ATTN_ERR_INVALID, eta.ATTN_ERR_UNSUPPORTED

BAD_CACHES = [
    (dict(d=12), UNSUPPORTED), (dict(d=264), UNSUPPORTED), (dict(page_size=4), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED),
    (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID), (dict(table_width=0), INVALID),
    (dict(table_width=1 << 27), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(table=0), INVALID), (dict(k=A + 8), INVALID), (dict(table=A + 2), INVALID),
    (dict(page_stride=8 * 16 * 128 + 4), INVALID), (dict(token_stride=120), INVALID),
    (dict(head_stride=0), INVALID), (dict(page_stride=-128), INVALID),
]


def paged(clib, cache=None, f16=False, **kw):
    a = dict(q=A, q_stride=32 * 128, cu=A, lens=A, o=A, lse=None, B=2, Hq=32, total=5, max_q=3,
             scale=0.1, window=0)
    a.update(kw)
    fn = clib.attn_paged_f16 if f16 else clib.attn_paged
    return fn(a["q"], a["q_stride"], cache if cache is not None else pages(), a["cu"], a["lens"],
              a["o"], a["lse"], a["B"], a["Hq"], a["total"], a["max_q"], a["scale"], a["window"],
              None)


def test_paged_refusals(clib):
    for kw, code in BAD_CACHES:
        assert paged(clib, pages(**kw)) == code, kw
    assert clib.attn_paged(A, 4096, None, A, A, A, None, 1, 32, 1, 1, 0.1, 0, None) == INVALID
    for kw in (dict(Hq=12), dict(Hq=0), dict(B=-1), dict(total=-1), dict(total=(1 << 29) + 1),
               dict(max_q=-1), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1),
               dict(q_stride=32 * 128 - 8), dict(q_stride=32 * 128 + 4), dict(q=None),
               dict(o=None), dict(cu=None), dict(lens=None), dict(q=A + 8), dict(o=A + 2),
               dict(lens=A + 2), dict(lse=A + 2)):
        assert paged(clib, **kw) == INVALID, kw
        assert paged(clib, f16=True, **kw) == INVALID, kw
    for kw in (dict(B=0), dict(total=0), dict(max_q=0)):  # nothing to do
        assert paged(clib, **kw) == eta.ATTN_OK, kw


def append(clib, cache=None, **kw):
    a = dict(q=A, qs=32 * 128, qo=A, qos=32 * 128, k=A, ks=1024, v=A, vs=1024, cu=A, lens=A,
             pos=None, turns=A, B=2, Hq=32, total=5, rot=128, amp=1.0)
    a.update(kw)
    return clib.attn_rope_append(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["v"],
                                 a["vs"], cache if cache is not None else pages(), a["cu"],
                                 a["lens"], a["pos"], a["turns"], a["B"], a["Hq"], a["total"],
                                 a["rot"], a["amp"], 0, None)


def test_append_refusals(clib):
    for kw, code in BAD_CACHES:
        assert append(clib, pages(**kw)) == code, kw
    for kw in (dict(rot=127), dict(rot=130), dict(rot=-2), dict(amp=float("inf")), dict(B=-1),
               dict(total=-1), dict(Hq=-1), dict(qs=4088), dict(ks=1020), dict(vs=1016),
               dict(qos=4100), dict(q=None), dict(qo=None), dict(k=None), dict(v=None),
               dict(cu=None), dict(lens=None), dict(turns=None), dict(turns=A + 4),
               dict(pos=A + 2), dict(k=A + 8), dict(Hq=70000)):
        assert append(clib, **kw) == INVALID, kw
    for kw in (dict(B=0), dict(total=0)):
        assert append(clib, **kw) == eta.ATTN_OK, kw


def rope(clib, strides=None, **kw):
    a = dict(q=A, qo=A, k=A, ko=A, pos=A, ps=0, turns=A, B=2, Hq=4, Hkv=2, N=8, d=64, rot=64,
             amp=1.0)
    a.update(kw)
    s = (ctypes.c_longlong * 12)(*(strides or [2048, 512, 64] * 4))
    return clib.attn_rope(a["q"], a["qo"], a["k"], a["ko"], s, a["pos"], a["ps"], a["turns"],
                          a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["rot"], a["amp"], 0, 0, None)


def test_rope_refusals(clib):
    assert rope(clib, d=60) == UNSUPPORTED and rope(clib, d=264) == UNSUPPORTED
    for kw in (dict(rot=63), dict(rot=66), dict(B=-1), dict(N=-1), dict(Hq=-1), dict(Hkv=-1),
               dict(amp=float("nan")), dict(q=None), dict(qo=None), dict(k=None), dict(ko=A + 8),
               dict(pos=None), dict(pos=A + 2), dict(ps=-1), dict(turns=None), dict(turns=A + 4),
               dict(B=1 << 16, N=1 << 16), dict(Hq=65535)):
        assert rope(clib, **kw) == INVALID, kw
    for i in range(12):
        s = [2048, 512, 64] * 4
        s[i] += 4
        assert rope(clib, s) == INVALID
        s[i] = -64
        assert rope(clib, s) == INVALID
    for kw in (dict(B=0), dict(N=0), dict(Hq=0, Hkv=0), dict(rot=0)):  # rot = 0 in place: a no-op
        assert rope(clib, **kw) == eta.ATTN_OK, kw


def update(clib, cache=None, layers=1, layer_stride=0, **kw):
    a = dict(lens=A, refs=A, source=A, add=A, table_out=2 * A, lens_out=2 * A, refs_out=2 * A,
             info=A, B=3)
    a.update(kw)
    c = cache if cache is not None else pages()
    return (clib.attn_pages_update(c, layers, layer_stride, a["lens"], a["refs"], a["source"],
                                   a["add"], a["table_out"], a["lens_out"], a["refs_out"],
                                   a["info"], a["B"], None),
            clib.attn_pages_compact(c, layers, layer_stride, a["lens"], a["refs"], a["table_out"],
                                    a["refs_out"], a["info"], a["B"], None))


def test_page_operation_refusals(clib):
    for kw, code in BAD_CACHES:
        assert update(clib, pages(**kw)) == (code, code), kw
    for kw in (dict(B=-1), dict(layers=0), dict(layer_stride=-8), dict(layer_stride=4),
               dict(lens=None), dict(refs=None), dict(table_out=None), dict(refs_out=None),
               dict(info=None), dict(lens=A + 2), dict(info=A + 1), dict(B=1 << 30),
               dict(table_out=A), dict(refs_out=A)):  # the last two: an output is its input
        assert update(clib, **kw) == (INVALID, INVALID), kw
    for kw in (dict(source=None), dict(add=None), dict(lens_out=None), dict(lens_out=A)):
        assert update(clib, **kw)[0] == INVALID, kw
    # a page's values have to lie in one piece
    for kw in (dict(head_stride=16 * 128 + 8), dict(token_stride=136), dict(page_stride=8 * 16 * 128 - 8)):
        assert update(clib, pages(**kw)) == (INVALID, INVALID), kw


def test_rope_turns_against_the_formulas(clib):
    i = np.arange(32)
    f = 10000.0 ** (-2 * i / 64)
    t, amp = eta.attn_rope_turns(64)
    assert amp == 1.0 and np.allclose(t.numpy(), f / (2 * math.pi), rtol=1e-14)
    t, amp = eta.attn_rope_turns(64, scaling="linear", factor=4)
    assert amp == 1.0 and np.allclose(t.numpy(), f / (8 * math.pi), rtol=1e-14)
    t, amp = eta.attn_rope_turns(64, scaling="base", factor=4)
    assert np.allclose(t.numpy(), (10000 * 4 ** (64 / 62)) ** (-2 * i / 64) / (2 * math.pi), rtol=1e-13)
    # parts: the first pairs unscaled, the last by the factor, never outside, falling
    t, amp = eta.attn_rope_turns(64, scaling="parts", factor=16, original=4096)
    g = t.numpy() * 2 * math.pi
    assert abs(amp - (0.1 * math.log(16) + 1)) < 1e-6
    assert np.allclose(g[:8], f[:8], rtol=1e-13) and np.allclose(g[-4:], f[-4:] / 16, rtol=1e-13)
    turns_made = 4096 * f / (2 * math.pi)
    assert np.allclose(g[turns_made > 40], f[turns_made > 40]) and (np.diff(g) < 0).all()
    # bands: by the turns over the original context, linear between 1 and 4
    t, amp = eta.attn_rope_turns(64, base=500000.0, scaling="bands", factor=8, original=8192)
    f5 = 500000.0 ** (-2 * i / 64)
    made = 8192 * f5 / (2 * math.pi)
    mix = np.clip((made - 1) / 3, 0, 1)
    assert amp == 1.0
    assert np.allclose(t.numpy() * 2 * math.pi, (1 - mix) * f5 / 8 + mix * f5, rtol=1e-13)


def test_rope_turns_refusals(clib):
    for kw in (dict(rot=0), dict(rot=7), dict(rot=258), dict(rot=64, base=1.0),
               dict(rot=64, base=float("nan")), dict(rot=64, scaling="linear", factor=0.5),
               dict(rot=2, scaling="base", factor=2.0),
               dict(rot=64, scaling="parts", factor=2, low=4, high=2),
               dict(rot=64, scaling="bands", factor=2, original=0.0)):
        with pytest.raises(eta.AttnError):
            eta.attn_rope_turns(**kw)
    with pytest.raises(ValueError):
        eta.attn_rope_turns(64, scaling="other")


def test_binding_refuses_cpu_tensors():
    kp, vp, table, refs = make_cache([20], 2, 64, 16, torch.bfloat16, 1)
    q = randn((3, 4, 64), torch.bfloat16, 2)
    with pytest.raises(ValueError):
        eta.attn_paged(q, kp, vp, table, cu([3]), torch.tensor([20], dtype=torch.int32))
    with pytest.raises(ValueError):
        eta.attn_rope(q[None], None, torch.arange(4, dtype=torch.int32), torch.zeros(4).double())
    with pytest.raises(ValueError):
        eta.attn_pages_compact(kp, vp, table, refs, refs)


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("window", [0, 5])
def test_oracle_paged_equals_contiguous(window):
    T, L = [1, 4, 7, 3], [9, 4, 20, 1]
    kp, vp, table, _ = make_cache(L, 2, 16, 8, torch.float16, 3)
    q = randn((sum(T) + 2, 6, 16), torch.float16, 4)
    c = cu(T)
    o, lse = ref.paged_attention_ref(q, kp, vp, table, c, L, 0.3, window)
    for b in range(4):
        for i in range(T[b]):
            at = L[b] - T[b] + i
            for h in range(6):
                js = [j for j in range(L[b]) if j <= at and (not window or j > at - window)]
                if not js:
                    assert (o[c[b] + i, h] == 0).all() and lse[c[b] + i, h] == -np.inf
                    continue
                k = np.stack([kp[table[b, j // 8], h // 3, j % 8].double().numpy() for j in js])
                v = np.stack([vp[table[b, j // 8], h // 3, j % 8].double().numpy() for j in js])
                s = 0.3 * k @ q[c[b] + i, h].double().numpy()
                p = np.exp(s - s.max())
                assert np.allclose(o[c[b] + i, h], p @ v / p.sum(), rtol=1e-12, atol=1e-14)
                assert abs(lse[c[b] + i, h] - (s.max() + math.log(p.sum()))) < 1e-12
    assert np.isnan(o[sum(T):]).all()  # rows of no sequence


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_is_a_rotation_with_its_transpose_as_gradient(interleaved):
    turns, amp = eta.attn_rope_turns(8)
    x, g = randn((3, 12), torch.float64, 5), randn((3, 12), torch.float64, 6)
    pos = np.array([0, 7, 100000])
    y = ref.rope_ref(x, pos, turns, 1.0, interleaved)
    assert np.allclose(y[0], x[0]) and np.allclose(y[:, 8:], x[:, 8:])
    assert np.allclose((y ** 2).sum(-1), (x.numpy() ** 2).sum(-1))
    assert np.allclose(ref.rope_ref(y, pos, turns, 1.0, interleaved, True), x)
    # the gradient of sum(g * rope(x)) by central differences
    dx = ref.rope_ref(g, pos, turns, 1.3, interleaved, True)
    loss = lambda z: float((ref.rope_ref(z, pos, turns, 1.3, interleaved) * g.numpy()).sum())  # noqa: E731
    for n in range(3):
        for c in range(12):
            e = np.zeros((3, 12))
            e[n, c] = 1e-4
            d = (loss(x.numpy() + e) - loss(x.numpy() - e)) / 2e-4
            assert abs(d - dx[n, c]) < 1e-8
    # scores depend on differences of positions only
    q, k = randn((12,), torch.float64, 7), randn((12,), torch.float64, 8)
    dot = lambda a, b: float((ref.rope_ref(q[None], [a], turns, 1.0, interleaved) *  # noqa: E731
                              ref.rope_ref(k[None], [b], turns, 1.0, interleaved)).sum())
    assert abs(dot(5, 3) - dot(1005, 1003)) < 1e-9


def test_oracle_update_keeps_every_row_whole():
    page, lens = 4, [9, 8, 0, 3, 6]
    kp, vp, table, refs = make_cache(lens, 1, 8, page, torch.float16, 9, spare=12, width=6)
    source, add = [1, 0, 0, -1, 4], [1, 0, 2, 5, 3]
    t, l, r, info, copies = ref.update_ref(table, lens, refs, source, add, page)
    assert info == [0, 0] and l == [9, 9, 11, 5, 9]
    k = kp.clone()
    for a, b in copies:
        k[b] = k[a]
    for b, s in enumerate(source):
        n = lens[s] if s >= 0 else 0
        if n:
            assert (ref.gather_cache(k, t[b], n) == ref.gather_cache(kp, table[s], n)).all()
    held = {}
    for b in range(5):
        for p in t[b][:-(-l[b] // page)]:
            held[p] = held.get(p, 0) + 1
        assert all(p == -1 for p in t[b][-(-l[b] // page):])
    assert all(r[p] == held.get(p, 0) for p in range(len(r)))
    # a page that a row will write on (behind its old length) is its own
    for b, s in enumerate(source):
        n = lens[s] if s >= 0 else 0
        for j in range(n // page, -(-l[b] // page)):
            assert held[t[b][j]] == 1
    # too few pages, or too long a row: nothing changes
    t2, l2, r2, info2, c2 = ref.update_ref(table, lens, refs, source, [1, 0, 2, 5, 60], page)
    assert info2[1] == 1 and c2 == [] and l2 == lens and r2 == refs.tolist()


def test_oracle_compact_keeps_every_row_whole():
    page, lens = 4, [9, 3, 0, 14]
    kp, _, table, refs = make_cache(lens, 2, 8, page, torch.float16, 10, spare=9, width=5)
    t, r, info, moves = ref.compact_ref(table, lens, refs, page)
    assert info == [8, len(moves)] and all(x > 0 for x in r[:8]) and not any(r[8:])
    assert all(a >= 8 > b for a, b in moves)
    k = kp.clone()
    for a, b in moves:
        k[b] = k[a]
    for b, l in enumerate(lens):
        assert (ref.gather_cache(k, t[b], l) == ref.gather_cache(kp, table[b], l)).all()


def test_error_bound_is_of_the_types_size():
    """The bound of the GPU comparison: some half steps of the type, not more."""
    L, T = [200], [3]
    kp, vp, table, _ = make_cache(L, 2, 64, 16, torch.bfloat16, 11)
    q = randn((3, 4, 64), torch.bfloat16, 12)
    o, _ = oracle.attention_ref(q.transpose(0, 1)[None], ref.gather_cache(kp.double(), table[0], 200)[None],
                                ref.gather_cache(vp.double(), table[0], 200)[None], 0.125, True)
    bo, bl = ref.paged_error_bound(q, kp, vp, table, cu(T), L, 0.125, 0, 2.0 ** -8, 2.0 ** -133)
    assert bo.max() < 2.2 * 2.0 ** -8 * 1.0 and bo.min() > 0  # sum p |v| < 1 here
    assert bl.max() < 2e-4
