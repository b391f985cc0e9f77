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
    over = np.abs(lse[bad] - rl[bad]) / (bl[bad] + 2.0 ** -23 * np.abs(rl[bad]))
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
    "chunk_page_512": ("bf16", 64, 4, 2, 512, [40, 1], [700, 1025], 0),
    "decode_page_1024": ("f16", 128, 8, 2, 1024, [1, 1], [1030, 5], 700),
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


def test_outputs_on_a_given_stream_keep_their_memory(lib):
    """Outputs that the call allocates for another stream are not handed out again, once
    dropped, before that stream is done with them."""
    T, L = [200], [30000]
    kp, vp, table, _ = make_cache(L, 2, 64, 64, torch.bfloat16, 51)
    q = randn((200, 8, 64), torch.bfloat16, 52)
    st = [x.cuda() for x in (q, kp, vp, table, cu(T), torch.tensor(L, dtype=torch.int32))]
    want, _ = lib.attn_paged(*st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = []
    for _ in range(30):
        lib.attn_paged(*st, stream=side)  # dropped at once
        keep.append(torch.zeros_like(want))  # would take its place, on the current stream
    torch.cuda.synchronize()
    assert not any(t.any() for t in keep)


def plain(q, kp, vp, table, T, L, scale, window, rows):
    """(which, o, lse, sum p |v|, sum of the visible |v|) in 64 bits on the GPU, of up to `rows` new
    tokens of each sequence (the first, the last, some between)."""
    Hq, d = q.shape[1:]
    Hkv, page = kp.shape[1], kp.shape[2]
    at, picked, out, ls, pv, av = 0, [], [], [], [], []
    for b, (t, l) in enumerate(zip(T, L)):
        if t:
            i = torch.linspace(0, t - 1, min(t, rows)).long().unique().cuda()
            ids = table[b, :-(-l // page)].long()
            j, pos = torch.arange(l, device="cuda"), l - t + i
            see = j[None] <= pos[:, None]
            if window:
                see &= j[None] > pos[:, None] - window
            ob = torch.zeros(len(i), Hq, d, dtype=torch.float64, device="cuda")
            wb, ab = torch.zeros_like(ob), torch.zeros_like(ob)
            lb = torch.full((len(i), Hq), -torch.inf, dtype=torch.float64, device="cuda")
            for h in range(Hq if l else 0):
                k = kp[ids, h // (Hq // Hkv)].reshape(-1, d)[:l].double()
                v = vp[ids, h // (Hq // Hkv)].reshape(-1, d)[:l].double()
                s = torch.where(see, q[at + i, h].double() @ k.T * scale, -torch.inf)
                lb[:, h] = torch.logsumexp(s, -1)
                some = torch.isfinite(lb[:, h])
                p = torch.exp(s[some] - lb[some, h, None])
                ob[some, h] = p @ v
                wb[some, h] = p @ v.abs()
                ab[some, h] = see[some].double() @ v.abs()
            pv.append(wb)
            av.append(ab)
            picked.append(at + i)
            out.append(ob)
            ls.append(lb)
        at += t
    return [torch.cat(x) for x in (picked, out, ls, pv, av)]


# The shapes on which the steps are dealt out in other ways: caches beyond L2 (chunks of items
# in step, rests to the other CTAs, whole items that begin anywhere), batches that a block or a
# kernel of its own plans, chunks of many tile pairs.
BIG = {
    "chunks_beyond_l2": ("bf16", 128, 8, 8, 64, [300], [20011], 0),
    "chunks_beyond_l2_group_4": ("bf16", 128, 32, 8, 128, [200, 1, 77], [17000, 9000, 300], 0),
    "chunks_beyond_l2_d64": ("f16", 64, 16, 16, 16, [257, 40], [30000, 12345], 0),
    "chunks_and_a_window": ("bf16", 128, 8, 8, 64, [300, 300], [20011, 5000], 3000),
    "whole_items_beyond_l2": ("bf16", 128, 8, 8, 128, [3000], [20000], 0),
    "whole_items_in_l2": ("f16", 64, 4, 2, 16, [5000, 33, 700], [5000, 900, 2000], 0),
    "long_chunk_of_many_pairs": ("bf16", 64, 32, 1, 64, [900], [2000], 0),
    "block_plan": ("bf16", 128, 8, 2, 16, [(7 * i) % 50 for i in range(90)], [60 + 13 * (i % 30) for i in range(90)], 0),
    "block_plan_beyond_l2": ("bf16", 128, 8, 8, 64, [40] * 34, [700 + 17 * i for i in range(34)], 0),
    "plan_kernel": ("f16", 64, 8, 1, 8, [(i * 5) % 7 for i in range(2500)], [6 + i % 20 for i in range(2500)], 0),
    "plan_kernel_beyond_l2": ("bf16", 128, 16, 8, 64, [20] + [1] * 2100, [9000] + [30] * 2100, 0),
    "decode_plan_kernel": ("bf16", 128, 8, 2, 16, [(i * 3) % 2 for i in range(3000)], [1 + i % 50 for i in range(3000)], 0),
    "decode_few_long": ("bf16", 128, 16, 2, 64, [1, 1], [60000, 33], 0),
    "few_tokens_long_window": ("f16", 128, 4, 1, 64, [8, 3], [30000, 200], 20000),
}


@pytest.mark.parametrize("name", BIG)
def test_large_caches_and_batches(lib, name):
    dtype, d, Hq, Hkv, page, T, L, window = BIG[name]
    dtype = DTYPES[dtype]
    n = [-(-l // page) for l in L]
    P, width = sum(n) + 5, max(n) + 1
    g = torch.Generator(device="cuda").manual_seed(len(name))
    kp = torch.randn(P, Hkv, page, d, device="cuda", generator=g).to(dtype)
    vp = torch.randn(P, Hkv, page, d, device="cuda", generator=g).to(dtype)
    ids = torch.randperm(P, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(L), width), -1, dtype=torch.int32)
    idc, at = ids.cpu(), 0
    for b, k in enumerate(n):
        table[b, :k] = idc[at:at + k]
        at += k
    used = torch.zeros(P, dtype=torch.bool, device="cuda")
    used[ids[:at].long()] = True
    kp[~used], vp[~used] = NAN, NAN
    table = table.cuda()
    q = torch.randn(sum(T), Hq, d, device="cuda", generator=g).to(dtype)
    args = (q, kp, vp, table, cu(T).cuda(), torch.tensor(L, dtype=torch.int32).cuda())
    o, lse = lib.attn_paged(*args, max_q=max(T), window=window)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
    scale = d ** -0.5
    rows, ro, rl, pv, av = plain(q, kp, vp, table, T, L, scale, window, 24)
    o64, l64 = o[rows].double(), lse[rows].double()
    assert torch.equal(torch.isneginf(l64), torch.isneginf(rl))
    # As in the oracle's bound: one rounding of the result, one of each probability (relative, or half
    # the type's smallest step against a sum of at least 1), and scores off by (d + 8) 2^-24 sum |q_c k_c|
    # scale < 2^-13, twice. (sum |q_c k_c| scale <= 15 for these values.)
    half = HALF_STEP[dtype]
    bound = half * ro.abs() * 1.01 + (half * 1.01 + 2.0 ** -12) * pv + LEAST[dtype] / 2 * av + LEAST[dtype]
    bad = ~((o64 - ro).abs() <= bound)
    assert not bad.any(), (rows[bad.any(-1).any(-1)].tolist(), bad.any(0).any(-1).nonzero().flatten().tolist(),
                           bad.sum().item(), ((o64 - ro).abs() / bound).max().item())
    seen = torch.isfinite(rl)
    assert ((l64 - rl).abs()[seen] <= 2.0 ** -13 + 2.0 ** -18).all()
    again, lse2 = lib.attn_paged(*args, max_q=max(T), window=window)
    assert torch.equal(o, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
def test_items_of_two_tiles_and_of_one_in_turns(lib, d):
    """Many short whole items, one after another in every CTA: two tiles of rows (whose output
    is staged), then one tile of two or three key tiles (whose groups exchange their sums)."""
    T = [64, 20] * 700
    L = [64 + 60 * (i % 3) for i in range(1400)]
    L = [l if t == 64 else 300 + l % 60 for t, l in zip(T, L)]
    kp, vp, table, _ = make_cache(L, 2, d, 64, torch.bfloat16, 41)
    q = randn((sum(T), 8, d), torch.bfloat16, 42)
    st = [x.cuda() for x in (q, kp, vp, table, cu(T), torch.tensor(L, dtype=torch.int32))]
    o, lse = lib.attn_paged(*st, max_q=64)
    rows, ro, rl, pv, av = plain(st[0], st[1], st[2], st[3], T, L, d ** -0.5, 0, 3)
    half = HALF_STEP[torch.bfloat16]
    assert ((o[rows].double() - ro).abs() <= half * ro.abs() * 1.01 + (half * 1.01 + 2.0 ** -12) * pv + 2.0 ** -30).all()
    assert ((lse[rows].double() - rl).abs() <= 2.0 ** -13 + 2.0 ** -18).all()
    for _ in range(20):
        again, lse2 = lib.attn_paged(*st, max_q=64)
        assert torch.equal(o, again) and torch.equal(lse, lse2)

@pytest.mark.parametrize("dtype, d, window", [("f16", 64, 0), ("f16", 64, 1024), ("bf16", 128, 0), ("bf16", 96, 300)])
def test_warps_without_rows_every_time(lib, dtype, d, window):
    """Row tiles with warps that have no row and warps that have some, first and second tiles of an
    item, whole items and cut ones, over many key tiles: the oracle's result, and the same bits
    whatever runs before and however cold the caches are. (A warp without rows once ran a step
    ahead of its tile's others, whose probabilities the product then missed.)"""
    dtype = DTYPES[dtype]
    T = [98, 34, 7, 241, 133, 83, 120, 59, 27]
    L = [1199, 3010, 917, 4437, 1362, 2307, 4195, 1067, 3552]
    kp, vp, table, _ = make_cache(L, 2, d, 16, dtype, 17, unused=NAN)
    q, c = randn((sum(T), 16, d), dtype, 18), cu(T)
    qd, kd, vd, td, cd = (x.cuda() for x in (q, kp, vp, table, c))
    ld = torch.tensor(L, dtype=torch.int32, device="cuda")

    def call():
        return lib.attn_paged(qd, kd, vd, td, cd, ld, max_q=max(T), window=window)

    o, lse = call()
    check(lib, o, lse, q, kp, vp, table, c, L, d ** -0.5, window)
    cold = torch.empty(1 << 26, dtype=torch.int32, device="cuda")  # larger than L2
    outs = []
    for i in range(60):
        if i % 3 == 0:
            cold.fill_(i)
        elif i % 3 == 1:  # another kernel's code in between
            cold[: 1 << 16].sort()
        outs.append(call())
    for o2, lse2 in outs:
        assert torch.equal(o2, o) and torch.equal(lse2, lse)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


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
