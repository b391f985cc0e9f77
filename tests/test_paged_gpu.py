"""Attention over a paged cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from paged_cases import DTYPES, HALF_STEP, LEAST, cu, make_cache, randn

pytestmark = pytest.mark.gpu

NAN = float("nan")


def attend(lib, q, kp, vp, table, c, L, **kw):
    dev = "cuda"
    Lt = torch.tensor(L, dtype=torch.int32)
    return lib.attn_paged(q.to(dev), kp.to(dev), vp.to(dev), table.to(dev), c.to(dev), Lt.to(dev), **kw)


def check(lib, o, lse, q, kp, vp, table, c, L, scale, window=0):
    """o and lse within the derived bound of the oracle's; pools without NaN in held places."""
    kz, vz = torch.nan_to_num(kp.float(), 0, 0, 0), torch.nan_to_num(vp.float(), 0, 0, 0)
    ro, rl = ref.paged_attention_ref(q, kz, vz, table, c, L, scale, window)
    bo, bl = ref.paged_error_bound(q, kz, vz, table, c, L, scale, window, HALF_STEP[q.dtype],
                                   LEAST[q.dtype])
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    rows = ~np.isnan(rl)
    assert np.isfinite(o[rows]).all()
    empty = np.isneginf(rl)
    assert (np.isneginf(lse) == empty)[rows].all()
    assert (o[empty] == 0).all()
    bad = rows & ~empty
    over = (np.abs(o - ro) / bo)[bad]
    assert over.max(initial=0) <= 1, f"o is {over.max():.2f} bounds off"
    over = (np.abs(lse - rl) / (bl + 2.0 ** -23 * np.abs(rl)))[bad]
    assert over.max(initial=0) <= 1, f"lse is {over.max():.2f} bounds off"
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


# dtype, d, Hq, Hkv, page, new tokens, cached tokens, window
CASES = {
    "one_token": ("bf16", 128, 8, 2, 16, [1], [1], 0),
    "decode_ragged": ("bf16", 128, 32, 8, 16, [1] * 7, [1, 15, 16, 17, 127, 129, 700], 0),
    "decode_f16_d64_page64": ("f16", 64, 8, 4, 64, [1] * 5, [64, 65, 128, 300, 1], 0),
    "decode_mha": ("bf16", 128, 3, 3, 32, [1] * 4, [200, 31, 33, 500], 0),
    "decode_mqa": ("f16", 128, 32, 1, 8, [1] * 3, [77, 1000, 8], 0),
    "decode_window": ("bf16", 128, 16, 4, 16, [1] * 4, [5, 128, 129, 900], 100),
    "empty_sequences": ("bf16", 128, 8, 2, 16, [0, 1, 0, 2, 0], [0, 0, 9, 40, 300], 0),
    "more_new_than_cached": ("f16", 64, 4, 2, 8, [5, 9, 300], [3, 0, 130], 0),
    "few_tokens": ("bf16", 128, 32, 8, 16, [2, 5, 8, 3], [100, 5, 300, 129], 0),
    "chunk_from_nothing": ("bf16", 128, 4, 4, 16, [300], [300], 0),
    "chunk_odd_group": ("bf16", 128, 15, 3, 16, [77, 133], [501, 133], 0),
    "chunk_group_7_d64": ("f16", 64, 14, 2, 32, [65, 3, 130], [900, 300, 131], 0),
    "chunk_over_long": ("bf16", 128, 8, 2, 128, [100], [3001], 0),
    "chunk_page_256": ("f16", 128, 8, 8, 256, [129, 1], [700, 513], 0),
    "chunk_page_8": ("bf16", 64, 8, 2, 8, [40, 200], [333, 200], 0),
    "chunk_window": ("bf16", 128, 8, 2, 16, [200, 64, 1], [1000, 64, 700], 130),
    "window_of_one": ("f16", 64, 8, 2, 16, [70, 1], [400, 129], 1),
    "group_128": ("bf16", 64, 128, 1, 16, [3, 1], [200, 129], 0),
    "group_33": ("bf16", 128, 33, 1, 16, [10], [260], 0),
    "d_96": ("bf16", 96, 8, 2, 16, [1, 60], [300, 400], 0),
    "d_80_f16": ("f16", 80, 4, 4, 32, [1, 17], [129, 40], 0),
    "d_32": ("bf16", 32, 8, 2, 16, [1, 90], [65, 190], 0),
    "d_8": ("f16", 8, 2, 1, 8, [1, 20], [65, 190], 0),
    "mixed_batch": ("bf16", 128, 16, 4, 64, [1, 1, 257, 1, 64, 0, 31], [900, 5, 600, 64, 64, 70, 31], 0),
    "many_short": ("bf16", 64, 4, 2, 16, [1] * 300, [1 + i % 40 for i in range(300)], 0),
    "generic_d_192": ("bf16", 192, 4, 2, 16, [1, 20, 0, 7], [100, 65, 5, 3], 0),
    "generic_d_256_window": ("f16", 256, 4, 1, 32, [33, 1], [90, 70], 20),
    "generic_group_160": ("bf16", 64, 160, 1, 16, [2], [70], 0),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_oracle(lib, name):
    dtype, d, Hq, Hkv, page, T, L, window = CASES[name]
    dtype = DTYPES[dtype]
    # What no sequence holds is NaN: pages behind the last, rows behind L.
    kp, vp, table, _ = make_cache(L, Hkv, d, page, dtype, len(name), unused=NAN)
    q = randn((sum(T), Hq, d), dtype, 100 + len(name))
    c = cu(T)
    o, lse = attend(lib, q, kp, vp, table, c, L, max_q=max(T), window=window)
    check(lib, o, lse, q, kp, vp, table, c, L, d ** -0.5, window)


def test_scale_and_defaults(lib):
    T, L = [3, 40], [50, 41]
    kp, vp, table, _ = make_cache(L, 2, 64, 16, torch.bfloat16, 1)
    q = randn((43, 4, 64), torch.bfloat16, 2)
    o, lse = attend(lib, q, kp, vp, table, cu(T), L, scale=0.37)
    check(lib, o, lse, q, kp, vp, table, cu(T), L, 0.37)
    o2, none = attend(lib, q, kp, vp, table, cu(T), L, scale=0.37, max_q=40, want_lse=False)
    assert none is None and torch.equal(o, o2)


def test_large_scores_and_a_moving_maximum(lib):
    """Scores of some hundreds, growing along the cache: the running maximum moves in every tile."""
    T, L = [1, 40], [1500, 900]
    kp, vp, table, _ = make_cache(L, 2, 128, 16, torch.bfloat16, 3)
    for b, l in enumerate(L):
        for t in range(l):
            kp[table[b, t // 16], :, t % 16] *= 0.5 + t / 300
    q = randn((41, 8, 128), torch.bfloat16, 4)
    o, lse = attend(lib, q, kp, vp, table, cu(T), L, max_q=40, scale=0.2)
    check(lib, o, lse, q, kp, vp, table, cu(T), L, 0.2)


@pytest.mark.parametrize("where", ["tokens_outermost", "interleaved", "wide_rows"])
@pytest.mark.parametrize("d", [64, 96, 192])
def test_strides(lib, where, d):
    T, L, page, Hkv, Hq = [1, 50], [200, 130], 16, 2, 6
    kp, vp, table, _ = make_cache(L, Hkv, d, page, torch.float16, 5)
    q, c = randn((51, Hq, d), torch.float16, 6), cu(T)
    kg, vg, qg = kp.cuda(), vp.cuda(), q.cuda()
    if where == "tokens_outermost":  # [page][row][head][d]
        kg, vg = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kg, vg))
    elif where == "interleaved":  # k and v of a page side by side
        both = torch.stack([kg, vg], 1)
        kg, vg = both[:, 0], both[:, 1]
    else:  # q is a part of a wider projection
        wide = torch.full((51, Hq + 4, d), NAN, dtype=torch.float16, device="cuda")
        wide[:, 2:2 + Hq] = qg
        qg = wide[:, 2:2 + Hq]
    o, lse = lib.attn_paged(qg, kg, vg, table.cuda(), c.cuda(), torch.tensor(L, dtype=torch.int32).cuda())
    check(lib, o, lse, q, kp, vp, table, c, L, d ** -0.5)


@pytest.mark.parametrize("d", [128, 192])
def test_rows_outside_every_sequence_are_left(lib, d):
    T, L = [2, 30], [40, 90]
    kp, vp, table, _ = make_cache(L, 2, d, 16, torch.bfloat16, 7)
    q = randn((40, 4, d), torch.bfloat16, 8)
    c = cu(T) + 3  # three rows before, five behind
    o = torch.full((40, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((40, 4), 7.0, device="cuda")
    attend(lib, q, kp, vp, table, c, L, max_q=30, o=o, lse=lse)
    check(lib, o, lse, q, kp, vp, table, c, L, d ** -0.5)
    for t in (o, lse):
        assert (t[:3] == 7).all() and (t[35:] == 7).all()


@pytest.mark.parametrize("d", [64, 256])
def test_bad_tables_are_reported_and_not_followed(lib, d):
    """A page id outside the pool, a length beyond the table, rows that decrease: an
    error status, the other sequences as always, and the context usable. (The ids are
    compared with the pool's size before any use, on the device.)"""
    T, L = [1, 1, 1], [40, 50, 60]
    kp, vp, table, _ = make_cache(L, 2, d, 16, torch.bfloat16, 9)
    q, c = randn((3, 4, d), torch.bfloat16, 10), cu([1, 1, 1])
    good, _ = attend(lib, q, kp, vp, table, c, L, max_q=1)
    bad = table.clone()
    bad[1, 1], bad[1, 2] = 1 << 30, -7
    o, _ = attend(lib, q, kp, vp, bad, c, L, max_q=1)
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2001)
    assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
    o, _ = attend(lib, q, kp, vp, table, c, [40, 1 << 20, 60], max_q=1)
    code, raw = lib.attn_get_device_status()
    assert code == lib.ATTN_ERR_PAGES and raw in (0x2001, 0x2002)
    assert torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
    attend(lib, q, kp, vp, table, torch.tensor([0, 3, 1, 9], dtype=torch.int32), L, max_q=1)
    assert lib.attn_get_device_status()[0] == lib.ATTN_ERR_PAGES
    o, _ = attend(lib, q, kp, vp, table, c, L, max_q=1)
    assert torch.equal(o, good) and lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_the_same_result_every_time_and_on_two_streams_at_once(lib):
    T, L = [1, 90, 1, 17], [2000, 700, 33, 400]
    sets = []
    for seed in (11, 12):
        kp, vp, table, _ = make_cache(L, 4, 128, 16, torch.bfloat16, seed)
        q = randn((sum(T), 16, 128), torch.bfloat16, seed + 10)
        sets.append([t.cuda() for t in (q, kp, vp, table, cu(T), torch.tensor(L, dtype=torch.int32))])
    first = [lib.attn_paged(*s, max_q=90) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(lib.attn_paged(*s, max_q=90))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(got):
        assert torch.equal(o, first[i % 2][0]) and torch.equal(lse, first[i % 2][1])
    # a stream given by argument, not the current one
    o, lse = lib.attn_paged(*sets[0], max_q=90, stream=streams[1])
    streams[1].synchronize()
    assert torch.equal(o, first[0][0])
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_two_captured_graphs_replayed_in_turn_and_together(lib):
    """Graphs of two batches, replayed after their lengths and queries changed in place."""
    T, L = [1, 1, 20], [500, 30, 300]
    graphs, state = [], []
    for seed in (21, 22):
        kp, vp, table, _ = make_cache([800] * 3, 2, 64, 16, torch.float16, seed)
        q = randn((22, 8, 64), torch.float16, seed + 10)
        st = [t.cuda() for t in (q, kp, vp, table, cu(T), torch.tensor(L, dtype=torch.int32))]
        o, lse = torch.empty_like(st[0]), torch.empty(22, 8, device="cuda")
        lib.attn_paged(*st, max_q=20, o=o, lse=lse)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.attn_paged(*st, max_q=20, o=o, lse=lse)
        graphs.append(g)
        state.append((st, o, lse))
    for step in range(3):
        for k, (st, o, lse) in enumerate(state):
            st[5].copy_(torch.tensor([500 + step, 30 + 90 * step, 300 - step], dtype=torch.int32))
            st[0].copy_(randn((22, 8, 64), torch.float16, 50 + 2 * step + k))
        torch.cuda.synchronize()
        side = [torch.cuda.Stream(), torch.cuda.Stream()]
        for g, s in zip(graphs, side):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for st, o, lse in state:
            want = lib.attn_paged(*st, max_q=20)
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_agrees_with_contiguous_prefill_and_packed_decode(lib):
    """The same attention through the library's other entry points."""
    N = 300
    kp, vp, table, _ = make_cache([N], 2, 128, 16, torch.bfloat16, 31)
    q = randn((N, 8, 128), torch.bfloat16, 32)
    k = torch.as_tensor(ref.gather_cache(kp.float(), table[0], N)).to(torch.bfloat16)[None]
    v = torch.as_tensor(ref.gather_cache(vp.float(), table[0], N)).to(torch.bfloat16)[None]
    o, lse = attend(lib, q, kp, vp, table, cu([N]), [N], max_q=N)
    oc, lc = lib.attn_fwd(q.transpose(0, 1).contiguous()[None].cuda(), k.cuda(), v.cuda(), causal=True)
    assert (o.float() - oc[0].transpose(0, 1).float()).abs().max() <= 2.0 ** -7 * oc.float().abs().max()
    assert (lse - lc[0].T).abs().max() < 1e-4
    o1, l1 = attend(lib, q[-1:].contiguous(), kp, vp, table, cu([1]), [N], max_q=1)
    od, ld = lib.attn_decode(q[-1:].contiguous().cuda(), k.reshape(-1).cuda(), v.reshape(-1).cuda(),
                             torch.tensor([N], dtype=torch.int32).cuda(), Hkv=2)
    assert (o1.float() - od.float()).abs().max() <= 2.0 ** -7 * od.float().abs().max()
    assert (l1 - ld).abs().max() < 1e-4


def test_binding_refusals(lib):
    kp, vp, table, _ = make_cache([20], 2, 64, 16, torch.bfloat16, 1)
    kg, vg, tg = kp.cuda(), vp.cuda(), table.cuda()
    q = randn((3, 4, 64), torch.bfloat16, 2).cuda()
    c, L = cu([3]).cuda(), torch.tensor([20], dtype=torch.int32).cuda()
    lib.attn_paged(q, kg, vg, tg, c, L)
    for args in ((q.half(), kg, vg, tg, c, L), (q, kg, vg[:, :1], tg, c, L), (q, kg, vg, tg.long(), c, L),
                 (q, kg, vg, tg, c.long(), L), (q, kg, vg, tg, c[:1], L), (q, kg, vg, tg, c, L.cpu()),
                 (q[..., :32], kg, vg, tg, c, L), (q, kg.float(), vg.float(), tg, c, L),
                 (q.transpose(0, 1), kg, vg, tg, c, L), (q, kg, vg.transpose(1, 2), tg, c, L)):
        with pytest.raises(ValueError):
            lib.attn_paged(*args)
    with pytest.raises(ValueError):
        lib.attn_paged(q, kg, vg, tg, c, L, o=torch.empty(3, 4, 32, device="cuda"))
    with pytest.raises(lib.AttnError):
        lib.attn_paged(q[:, :3].contiguous(), kg, vg, tg, c, L)  # 3 heads over 2
