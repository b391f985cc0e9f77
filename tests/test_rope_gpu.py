"""Rotary positions and their append to the paged cache against the fp64 oracle."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from paged_cases import DTYPES, HALF_STEP, LEAST, cu, make_cache, randn

pytestmark = pytest.mark.gpu


def near(y, want, x, rot, interleaved, amp):
    """|y - want| within one rounding of want, and 2^-21 of the pair for the 32-bit
    rotation: cosine and sine are off by 2 pi 2^-25 + 2^-23 at most, the three
    products and sums by 2^-24 each, relative to amp (|x_a| + |x_b|)."""
    y, want, x = y.double().cpu().numpy(), np.asarray(want), x.double().cpu().numpy()
    size = np.abs(x).copy()
    h = rot // 2
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, h), slice(h, rot))
    both = np.abs(x[..., a]) + np.abs(x[..., b])
    size[..., a], size[..., b] = both, both
    size[..., rot:] = 0
    return np.abs(y - want), lambda t: HALF_STEP[t] * np.abs(want) * (1 + 2.0 ** -8) + \
        size * amp * 2.0 ** -21 + LEAST[t]


def assert_near(y, want, x, rot, interleaved, amp, dtype):
    err, bound = near(y, want, x, rot, interleaved, amp)
    over = (err / bound(dtype)).max(initial=0)
    assert over <= 1, f"{over:.2f} bounds off"


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 128), ("f16", 64, 32), ("bf16", 64, 48),
                                         ("f16", 80, 20), ("bf16", 256, 256), ("f16", 256, 16),
                                         ("bf16", 8, 2), ("f16", 96, 0), ("bf16", 104, 64), ("f16", 64, 62)])
def test_against_the_oracle(lib, dtype, d, rot, interleaved, backward):
    dt = DTYPES[dtype]
    turns, amp = lib.attn_rope_turns(rot, scaling="parts", factor=4) if rot else (torch.zeros(0).double(), 1.5)
    for B, Hq, Hkv, N in ((2, 5, 2, 13), (1, 1, 1, 1), (3, 33, 0, 7)):
        q = randn((B, Hq, N, d), dt, d + rot)
        k = randn((B, Hkv, N, d), dt, d + rot + 1) if Hkv else None
        pos = torch.randint(-5, 2000, (B, N), dtype=torch.int32, generator=torch.Generator().manual_seed(3))
        fn = lib.attn_rope_bwd if backward else lib.attn_rope
        qo, ko = fn(q.cuda(), k.cuda() if Hkv else None, pos.cuda(), turns.cuda(), amp=amp,
                    interleaved=interleaved)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                assert y is None
                continue
            want = ref.rope_ref(x, pos[:, None].numpy(), turns, amp, interleaved, backward)
            assert_near(y, want, x, rot, interleaved, amp, dt)
            assert torch.equal(y[..., rot:].cpu(), x[..., rot:])  # passes through
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_far_positions_lose_nothing(lib):
    turns, amp = lib.attn_rope_turns(128)
    pos = torch.tensor([0, 1, 131071, 1 << 20, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    q = randn((1, 3, 6, 128), torch.float16, 1)
    qo, _ = lib.attn_rope(q.cuda(), None, pos.cuda(), turns.cuda())
    # turns are held in 64 bits: at 2^31 positions they are off by 2^31 2^-53 of a turn, as in the oracle
    assert_near(qo, ref.rope_ref(q, pos.numpy(), turns, 1.0, False), q, 128, False, 1.0, torch.float16)


def test_in_place_strided_and_shared_positions(lib):
    turns, amp = lib.attn_rope_turns(64)
    B, N, H = 2, 37, 6
    pos = torch.arange(100, 100 + N, dtype=torch.int32).cuda()
    rows = randn((B, N, H + 4, 96), torch.bfloat16, 2)  # tokens outermost: [B, N, heads, d]
    g = rows.cuda()
    q, k = g[:, :, :H].transpose(1, 2), g[:, :, H:H + 2].transpose(1, 2)
    want = [ref.rope_ref(x.cpu(), pos.cpu().numpy(), turns, 1.0, True) for x in (q, k)]
    before = [x.cpu().clone() for x in (q, k)]
    new = lib.attn_rope(q, k, pos, turns.cuda(), interleaved=True)
    for y, w, x in zip(new, want, before):
        assert_near(y, w, x, 64, True, 1.0, torch.bfloat16)
    q2, k2 = lib.attn_rope(q, k, pos, turns.cuda(), interleaved=True, q_out=q, k_out=k)
    assert q2.data_ptr() == q.data_ptr()
    assert torch.equal(q, new[0]) and torch.equal(k, new[1])
    assert torch.equal(g[:, :, H + 2:].cpu(), rows[:, :, H + 2:])  # the rest of the rows is untouched
    assert torch.equal(g[..., 64:].cpu(), rows[..., 64:])


def test_gradient_against_differences(lib):
    """d/dx sum(g rope(x)) by differences of the kernel itself, in steps that bf16 and the sum can tell."""
    turns, amp = lib.attn_rope_turns(16)
    pos = torch.tensor([3, 500], dtype=torch.int32).cuda()
    x = torch.zeros(1, 1, 2, 24, dtype=torch.float16)
    g = randn((1, 1, 2, 24), torch.float16, 4)
    dx, _ = lib.attn_rope_bwd(g.cuda(), None, pos, turns.cuda(), amp=1.25)
    for n in range(2):
        for c in range(24):
            e = x.clone()
            e[0, 0, n, c] = 1.0  # the map is linear: the difference quotient is exact at any step
            y, _ = lib.attn_rope(e.cuda(), None, pos, turns.cuda(), amp=1.25)
            d = float((y.double().cpu() * g.double()).sum())
            # y has two values of at most 1.25, each rounded by 2^-11; dx is rounded once
            size = float(g[0, 0, n].abs().max())
            assert abs(d - float(dx[0, 0, n, c])) <= 2.0 ** -11 * (2 * 1.25 * size + abs(d)) + 1e-6


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,rot,page,Hq,Hkv", [
    ("bf16", 128, 128, 16, 8, 2), ("f16", 64, 32, 64, 4, 4), ("bf16", 96, 0, 8, 6, 1),
    ("f16", 192, 64, 32, 3, 3), ("bf16", 64, 20, 16, 2, 1)])
@pytest.mark.parametrize("T,L", [([1] * 5, [1, 16, 17, 300, 64]), ([0, 7, 40, 0, 1, 3], [9, 7, 100, 0, 33, 1])])
def test_append_against_the_oracle(lib, T, L, dtype, d, rot, page, Hq, Hkv, interleaved):
    dt = DTYPES[dtype]
    kp, vp, table, _ = make_cache(L, Hkv, d, page, dt, 5)
    total = sum(T) + 2
    qkv = randn((total, Hq + 2 * Hkv, d), dt, 6)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    turns, amp = lib.attn_rope_turns(rot, scaling="bands", factor=8, original=64.0) if rot else \
        (torch.zeros(0).double(), 1.0)
    c, Lt = cu(T), torch.tensor(L, dtype=torch.int32)
    for pos in (None, torch.arange(5, 5 + total, dtype=torch.int32) * 3):
        kg, vg, g = kp.cuda(), vp.cuda(), qkv.cuda()
        qo = lib.attn_rope_append(g[:, :Hq], g[:, Hq:Hq + Hkv], g[:, Hq + Hkv:], kg, vg, table.cuda(),
                                  c.cuda(), Lt.cuda(), turns.cuda(), amp=amp, interleaved=interleaved,
                                  pos=None if pos is None else pos.cuda())
        wq, wk, wv = ref.append_ref(q, k, v, kp, vp, table, c, L, turns, amp, interleaved, pos)
        n = sum(T)
        assert_near(qo[:n], wq[:n], q[:n], rot, interleaved, amp, dt)
        assert torch.equal(vg.double().cpu(), torch.from_numpy(wv))
        # keys: written places within the bound, all others untouched
        kd = kg.double().cpu().numpy()
        touched = (wk != kp.double().numpy())
        size = float(qkv.abs().max()) * 2 * amp
        bound = HALF_STEP[dt] * np.abs(wk) * (1 + 2.0 ** -8) + size * 2.0 ** -21 + LEAST[dt]
        assert (np.abs(kd - wk) <= bound * touched).all()
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK


def test_append_with_more_new_tokens_than_positions_and_bad_pages(lib):
    T, L = [6, 2], [4, 20]
    kp, vp, table, _ = make_cache(L, 2, 64, 16, torch.bfloat16, 7)
    qkv = randn((8, 6, 64), torch.bfloat16, 8)
    turns, _ = lib.attn_rope_turns(64)
    c, Lt = cu(T).cuda(), torch.tensor(L, dtype=torch.int32).cuda()
    kg, vg, g = kp.cuda(), vp.cuda(), qkv.cuda()
    lib.attn_rope_append(g[:, :2], g[:, 2:4], g[:, 4:], kg, vg, table.cuda(), c, Lt, turns.cuda())
    _, wk, wv = ref.append_ref(qkv[:, :2], qkv[:, 2:4], qkv[:, 4:], kp, vp, table, cu(T), L, turns, 1.0, False)
    assert torch.equal(vg.double().cpu(), torch.from_numpy(wv))  # positions -2, -1 are not stored
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
    bad = table.clone()
    bad[1, 1] = kp.shape[0]  # positions 18, 19 of sequence 1
    kg, vg = kp.cuda(), vp.cuda()
    lib.attn_rope_append(g[:, :2], g[:, 2:4], g[:, 4:], kg, vg, bad.cuda(), c, Lt, turns.cuda())
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2001)
    wv[table[1, 1]] = vp[table[1, 1]].double().numpy()  # nothing of them was stored
    assert torch.equal(vg.double().cpu(), torch.from_numpy(wv))


def test_many_sequences_find_their_rows(lib):
    """Sequence look-up over many and empty sequences (rounds of 32 pivots)."""
    g = torch.Generator().manual_seed(9)
    T = torch.randint(0, 3, (2500,), generator=g).tolist()
    L = [max(t, 1) + int(x) for t, x in zip(T, torch.randint(0, 9, (2500,), generator=g))]
    kp, vp, table, _ = make_cache(L, 1, 16, 8, torch.float16, 10)
    total = sum(T)
    v = randn((total, 1, 16), torch.float16, 11)
    turns = torch.zeros(0, dtype=torch.float64).cuda()
    kg, vg = kp.cuda(), vp.cuda()
    lib.attn_rope_append(v.cuda(), v.cuda(), v.cuda(), kg, vg, table.cuda(), cu(T).cuda(),
                         torch.tensor(L, dtype=torch.int32).cuda(), turns)
    at = 0
    for b, (t, l) in enumerate(zip(T, L)):
        for i in range(t):
            p = l - t + i
            vp[table[b, p // 8], :, p % 8] = v[at]
            at += 1
    assert torch.equal(vg.cpu(), vp)


def test_capture_and_other_streams(lib):
    turns, _ = lib.attn_rope_turns(64)
    tg = turns.cuda()
    q = randn((1, 4, 50, 64), torch.bfloat16, 12).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda()
    want, _ = lib.attn_rope(q, None, pos, tg)
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.attn_rope(q, None, pos, tg, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got, _ = lib.attn_rope(q, None, pos, tg)
    s.synchronize()
    assert torch.equal(got, want)


def test_binding_refusals(lib):
    q = randn((1, 2, 3, 64), torch.bfloat16, 1).cuda()
    pos = torch.arange(3, dtype=torch.int32).cuda()
    turns = lib.attn_rope_turns(64)[0].cuda()
    for args in ((q.float(), None, pos, turns), (q[0], None, pos, turns), (q, q[:, :, :2], pos, turns),
                 (q, q.half(), pos, turns), (q, None, pos.long(), turns), (q, None, pos[:2], turns),
                 (q, None, pos, turns.float()), (q, None, pos, torch.zeros(33).double().cuda()),
                 (q.transpose(2, 3), None, pos, turns), (q, None, pos.cpu(), turns)):
        with pytest.raises(ValueError):
            lib.attn_rope(*args)
