"""Page update and compaction against the row-by-row oracle, and a run of all paged operators together."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from paged_cases import HALF_STEP, LEAST, cu, make_cache, randn

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def check_update(lib, kp, vp, table, lens, refs, source, add, page, order=None):
    P0 = kp.dim() - 4  # layers in front?
    kg, vg = kp.cuda(), vp.cuda()
    if order == "tokens_outermost":
        kg, vg = (x.transpose(-3, -2).contiguous().transpose(-3, -2) for x in (kg, vg))
    t, l, r, info = lib.attn_pages_update(kg, vg, table.cuda(), ints(lens), refs.cuda(), ints(source), ints(add))
    wt, wl, wr, winfo, copies = ref.update_ref(table, lens, refs, source, add, page)
    assert info.tolist() == winfo
    assert l.tolist() == wl and r.tolist() == wr and t.tolist() == wt
    wk, wv = kp.clone(), vp.clone()
    for a, b in copies:
        for pool in (wk, wv):
            pool.select(P0, b).copy_(pool.select(P0, a))
    assert torch.equal(kg.cpu(), wk) and torch.equal(vg.cpu(), wv)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
    return wt, wl, wr


CASES = {
    "grow": ([5, 16, 0, 31], [0, 1, 2, 3], [1, 1, 1, 1]),
    "free_all": ([5, 16, 0, 31], [-1] * 4, [0] * 4),
    "fork_to_all": ([21, 3, 40, 8], [0, 0, 0, 0], [1, 2, 3, 40]),
    "fork_of_another_row": ([21, 3, 40, 8], [2, 2, 1, 1], [1, 1, 1, 1]),
    "swap": ([21, 3, 40, 16], [3, 2, 1, 0], [1, 1, 1, 1]),
    "full_pages_only": ([16, 32, 48, 0], [1, 1, 1, 2], [0, 1, 16, 17]),
    "new_ones": ([0, 0, 9, 0], [-1, -1, 2, -1], [33, 0, 7, 16]),
    "nothing": ([21, 3, 40, 8], [0, 1, 2, 3], [0, 0, 0, 0]),
    "negative_growth_is_none": ([21, 3, 40, 8], [0, 0, 2, 3], [-5, -1, 0, -100]),
}


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("name", CASES)
def test_update(lib, name, layers):
    lens, source, add = CASES[name]
    kp, vp, table, refs = make_cache(lens, 2, 8, 16, torch.bfloat16, 1, spare=14, width=8, layers=layers)
    check_update(lib, kp, vp, table, lens, refs, source, add, 16)
    check_update(lib, kp, vp, table, lens, refs, source, add, 16, "tokens_outermost")


@pytest.mark.parametrize("B,page,seed", [(1, 8, 1), (7, 8, 2), (33, 64, 3), (100, 16, 4), (1500, 8, 5), (1700, 64, 6)])
def test_update_random_steps(lib, B, page, seed):
    """Several steps one after another: shared pages, forks of forks, ends and starts."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, 60, B).tolist()
    kp, vp, table, refs = make_cache(lens, 1, 8, page, torch.float16, seed, spare=B * 30 + 20, width=40)
    for step in range(4):
        source = [int(rng.integers(0, B)) if x < 0.4 else -1 if x < 0.5 else b
                  for b, x in enumerate(rng.random(B))]
        add = rng.integers(0, 25, B).tolist()
        t, l, r = check_update(lib, kp, vp, table, lens, refs, source, add, page)
        table, lens, refs = torch.tensor(t, dtype=torch.int32), l, torch.tensor(r, dtype=torch.int32)


def test_update_refuses_what_does_not_fit_and_changes_nothing(lib):
    lens = [21, 3, 40, 8]
    kp, vp, table, refs = make_cache(lens, 2, 8, 16, torch.bfloat16, 3, spare=2, width=4)
    for source, add, info in (([0, 0, 0, 0], [40, 40, 40, 40], None), ([0, 1, 2, 3], [1, 1, 30, 0], [0, 1])):
        want = ref.update_ref(table, lens, refs, source, add, 16)
        assert want[3] != [0, 0] and (info is None or want[3] == info)
        check_update(lib, kp, vp, table, lens, refs, source, add, 16)


def test_update_pinned_pages_and_bad_sources(lib):
    lens = [21, 3]
    kp, vp, table, refs = make_cache(lens, 2, 8, 16, torch.bfloat16, 4, spare=6, width=4)
    refs[int(table[0, 0])] += 1  # held from outside: stays when its row ends
    check_update(lib, kp, vp, table, lens, refs, [-1, -1], [0, 0], 16)
    lib.attn_pages_update(kp.cuda(), vp.cuda(), table.cuda(), ints(lens), refs.cuda(), ints([2, 0]), ints([0, 0]))
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2004)
    bad = table.clone()
    bad[0, 1] = 1 << 29
    lib.attn_pages_update(kp.cuda(), vp.cuda(), bad.cuda(), ints(lens), refs.cuda(), ints([1, 0]), ints([0, 0]))
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2001)
    lib.attn_pages_update(kp.cuda(), vp.cuda(), table.cuda(), ints([21, 900]), refs.cuda(), ints([0, 1]),
                          ints([0, 0]))
    assert lib.attn_get_device_status()[0] == lib.ATTN_ERR_PAGES


@pytest.mark.parametrize("layers", [None, 2])
@pytest.mark.parametrize("lens,page,spare,seed", [
    ([5, 16, 0, 31], 8, 0, 1), ([5, 16, 0, 31], 8, 1, 2), ([5, 16, 0, 31], 8, 50, 3), ([], 8, 9, 4),
    ([0, 0], 16, 5, 5), ([300] * 20, 16, 9000, 6), ([1] * 900, 8, 20000, 7), ([700, 20], 64, 3, 8),
    ([9] * 700, 8, 30000, 9), ([40] * 1000, 8, 10, 10)])
def test_compact(lib, lens, page, spare, seed, layers):
    kp, vp, table, refs = make_cache(lens, 1, 8, page, torch.float16, seed, spare=spare, layers=layers)
    if len(lens) > 2:  # two rows that share a page
        table[1, 0] = table[0, 0]
        refs = torch.zeros_like(refs)
        for b, l in enumerate(lens):
            for j in range(-(-l // page)):
                refs[table[b, j]] += 1
    if len(refs) > 4:
        refs[2] += 1  # and one held from outside
    kg, vg = kp.cuda(), vp.cuda()
    t, r, info = lib.attn_pages_compact(kg, vg, table.cuda(), ints(lens), refs.cuda())
    wt, wr, winfo, moves = ref.compact_ref(table, lens, refs, page)
    assert info.tolist() == winfo and r.tolist() == wr and t.tolist() == wt
    at = 1 if layers else 0
    for a, b in moves:
        for pool in (kp, vp):
            pool.select(at, b).copy_(pool.select(at, a))
    assert torch.equal(kg.cpu(), kp) and torch.equal(vg.cpu(), vp)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_large_pages_and_layer_views(lib):
    """Pages of several copy pieces with a ragged last one, pools that are views of a bigger buffer."""
    lens = [100, 300, 17]
    kp, vp, table, refs = make_cache(lens, 5, 72, 128, torch.bfloat16, 5, spare=9, layers=3)
    both = torch.stack([kp, vp], 2).cuda()  # [layers, P, 2, Hkv, page, d]
    kg, vg = both[:, :, 0], both[:, :, 1]
    t, l, r, info = lib.attn_pages_update(kg, vg, table.cuda(), ints(lens), refs.cuda(), ints([1, 1, 1]),
                                          ints([1, 0, 1]))
    wt, wl, wr, winfo, copies = ref.update_ref(table, lens, refs, [1, 1, 1], [1, 0, 1], 128)
    assert t.tolist() == wt and r.tolist() == wr and len(copies) == 2
    for a, b in copies:
        kp[:, b], vp[:, b] = kp[:, a], vp[:, a]
    assert torch.equal(kg.cpu(), kp) and torch.equal(vg.cpu(), vp)


def test_offsets_beyond_32_bits(lib):
    """Pages more than 2^31 values apart (one layer of a pool with all layers side by side):
    append, attention of one token and of a chunk, update and compaction."""
    lens, page, Hkv, d, Hq = [40, 100], 16, 2, 64, 4
    kp, vp, table, refs = make_cache(lens, Hkv, d, page, torch.bfloat16, 8, spare=6, width=9)
    P, n = kp.shape[0], Hkv * page * d
    wide = (1 << 32) // (P - 2) // 8 * 8  # values between pages: the last ones lie behind 2^32
    big = torch.empty((P - 1) * wide + 2 * n, dtype=torch.bfloat16, device="cuda")
    view = lambda at: big.as_strided((P, Hkv, page, d), (wide, page * d, d, 1), at)  # noqa: E731
    kg, vg = view(0), view(n)
    kg.copy_(kp)
    vg.copy_(vp)
    kd, vd = kp.cuda(), vp.cuda()
    turns = lib.attn_rope_turns(64)[0].cuda()
    for T in ([1, 1], [30, 90]):
        x = randn((sum(T), Hq + 2 * Hkv, d), torch.bfloat16, 9).cuda()
        got = []
        for k, v in ((kg, vg), (kd, vd)):
            q = lib.attn_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], k, v, table.cuda(), cu(T).cuda(),
                                     ints(lens), turns)
            got.append((q, *lib.attn_paged(q, k, v, table.cuda(), cu(T).cuda(), ints(lens), max_q=max(T))))
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert torch.equal(kg, kd) and torch.equal(vg, vd)
    for k, v in ((kg, vg), (kd, vd)):
        out = lib.attn_pages_update(k, v, table.cuda(), ints(lens), refs.cuda(), ints([1, 1]), ints([1, 20]))
        got.append(out + lib.attn_pages_compact(k, v, out[0], out[1], out[2]))
    assert all(torch.equal(a, b) for a, b in zip(got[2], got[3]))
    assert torch.equal(kg, kd) and torch.equal(vg, vd) and int(got[2][6][1]) >= 0
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_capture_two_graphs_and_streams(lib):
    lens = [21, 3, 40, 8]
    kp, vp, table, refs = make_cache(lens, 2, 8, 16, torch.bfloat16, 6, spare=20, width=8)
    source, add = ints([2, 2, 1, 3]), ints([1, 1, 1, 1])
    outs, graphs = [], []
    for _ in range(2):
        kg, vg = kp.cuda(), vp.cuda()
        st = (table.cuda(), ints(lens), refs.cuda())
        out = dict(table_out=torch.zeros_like(st[0]), lens_out=torch.zeros_like(st[1]),
                   refs_out=torch.zeros_like(st[2]), info=torch.zeros(2, dtype=torch.int32, device="cuda"))
        lib.attn_pages_update(kg, vg, *st, source, add, **out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lib.attn_pages_update(kg, vg, *st, source, add, **out)
        for t in out.values():
            t.zero_()
        graphs.append((g, kg, vg, st))
        outs.append(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for (g, *_), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    wt, wl, wr, winfo, _ = ref.update_ref(table, lens, refs, [2, 2, 1, 3], [1] * 4, 16)
    for out in outs:
        assert out["table_out"].tolist() == wt and out["lens_out"].tolist() == wl
        assert out["refs_out"].tolist() == wr and out["info"].tolist() == winfo


def test_binding_refusals(lib):
    kp, vp, table, refs = make_cache([20, 5], 2, 8, 16, torch.bfloat16, 1)
    kg, vg, t, r = kp.cuda(), vp.cuda(), table.cuda(), refs.cuda()
    L = ints([20, 5])
    for args in ((kg, vg, t, L, r[:-1]), (kg, vg, t, L.long(), r), (kg, vg, t[:, ::2], L, r), (kg, kg[1:], t, L, r)):
        with pytest.raises(ValueError):
            lib.attn_pages_compact(*args)
    for kw in (dict(table_out=t), dict(refs_out=r)):
        with pytest.raises(lib.AttnError):
            lib.attn_pages_compact(kg, vg, t, L, r, **kw)
    with pytest.raises(lib.AttnError):
        lib.attn_pages_update(kg, vg, t, L, r, L, L, lens_out=L)


def test_a_serving_run_of_all_of_them(lib):
    """Prompts in chunks, decode steps, forks, an end, a new prompt, a compaction: every
    step's attention is that of the tokens that each row has seen, kept apart on the host."""
    dt, Hq, Hkv, d, page, B, width = torch.bfloat16, 4, 2, 64, 16, 4, 12
    P = 60
    g = torch.Generator().manual_seed(77)
    kg = torch.full((P, Hkv, page, d), float("nan"), dtype=dt, device="cuda")
    vg = kg.clone()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(P, dtype=torch.int32, device="cuda")
    turns, amp = lib.attn_rope_turns(32, scaling="parts", factor=4, original=64)
    tg = turns.cuda()
    seen = [[] for _ in range(B)]  # (k, v) rounded rows, as the cache holds them
    steps = [([-1, -1, -1, -1], [40, 17, 1, 0]), ([0, 1, 2, -1], [30, 1, 1, 5]), ([0, 1, 1, 3], [1, 1, 1, 1]),
             ([0, 2, 2, 2], [1, 1, 1, 1]), ([3, 1, -1, 3], [1, 1, 20, 1]), ([0, 1, 2, 3], [1, 1, 1, 1])]
    for n, (source, add) in enumerate(steps):
        table, lens, refs, info = lib.attn_pages_update(kg, vg, table, lens, refs, ints(source), ints(add))
        assert info.tolist() == [0, 0]
        if n in (3, 5):
            table, refs, info = lib.attn_pages_compact(kg, vg, table, lens, refs)
            assert info[0] == (refs > 0).sum() and not (refs[int(info[0]):] > 0).any()
        c = cu(add)
        qkv = torch.randn((sum(add), Hq + 2 * Hkv, d), generator=g).to(dt)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        x = qkv.cuda()
        qr = lib.attn_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kg, vg, table, c.cuda(), lens, tg,
                                  amp=amp)
        o, lse = lib.attn_paged(qr, kg, vg, table, c.cuda(), lens, max_q=max(add))
        assert lib.attn_get_device_status()[0] == lib.ATTN_OK
        seen = [list(seen[s]) if s >= 0 else [] for s in source]
        qr = qr.cpu()
        for b in range(B):
            for i in range(add[b]):
                row, at = int(c[b]) + i, len(seen[b])
                kr = torch.from_numpy(ref.rope_ref(k[row], np.full(Hkv, at), turns, amp, False))
                held = kg[int(table[b, at // page]), :, at % page].cpu()
                assert ((held.double() - kr).abs() <= 2.0 ** -8 * kr.abs() * 1.01 + 2.0 ** -18).all()
                seen[b].append((held, v[row]))
            assert len(seen[b]) == int(lens[b])
            if add[b] == 0:
                continue
            kk = torch.stack([a for a, _ in seen[b]], 1)[None]  # [1, Hkv, L, d]
            vv = torch.stack([a for _, a in seen[b]], 1)[None]
            part = slice(int(c[b]), int(c[b + 1]))
            one = kk[0].transpose(0, 1).reshape(-1, 1, Hkv, d).transpose(1, 2)  # pages of one token
            two = vv[0].transpose(0, 1).reshape(-1, 1, Hkv, d).transpose(1, 2)
            ids = torch.arange(len(seen[b]), dtype=torch.int32)[None]
            args = (qr[part], one, two, ids, cu([add[b]]), [len(seen[b])], d ** -0.5, 0)
            wo, wl = ref.paged_attention_ref(*args)
            bo, bl = ref.paged_error_bound(*args, HALF_STEP[dt], LEAST[dt])
            assert (np.abs(o[part].double().cpu().numpy() - wo) <= bo).all(), (n, b)
            assert (np.abs(lse[part].double().cpu().numpy() - wl) <= bl + 2.0 ** -23 * np.abs(wl)).all()
