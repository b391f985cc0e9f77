"""Attention over a paged cache with infinite and NaN values at keys that tokens see."""
import pytest
import torch

from paged_cases import DTYPES, HALF_STEP, LEAST, cu, make_cache, randn

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")

# dtype, d, Hq, Hkv, page, new tokens, cached tokens, window. Few long sequences are cut
# between CTAs, many short ones are not.
CASES = {
    "decode_cut": ("bf16", 128, 8, 2, 16, [1, 1], [9000, 700], 0),
    "decode_whole": ("f16", 128, 8, 2, 16, [1] * 200, [60 + i for i in range(200)], 0),
    "decode_window_d64": ("f16", 64, 8, 4, 64, [1, 1, 1], [3000, 1500, 90], 1000),
    "few_tokens_cut": ("bf16", 128, 32, 8, 16, [4, 7], [5000, 300], 0),
    "decode_group_32": ("bf16", 128, 32, 1, 16, [1, 1], [4000, 60], 0),
    "tiles_cut": ("bf16", 128, 8, 2, 16, [90, 300], [3000, 300], 0),
    "tiles_cut_d64": ("f16", 64, 16, 2, 16, [133, 40], [4000, 900], 0),
    "tiles_whole": ("bf16", 128, 4, 4, 32, [130] * 60, [150 + i for i in range(60)], 0),
    "tiles_window": ("bf16", 128, 8, 2, 16, [200, 64], [1500, 64], 333),
    "one_tile_whole": ("bf16", 64, 8, 2, 64, [20] * 300, [300 + i % 60 for i in range(300)], 0),
    "chunks_beyond_l2": ("bf16", 128, 8, 8, 64, [300], [20011], 0),
    "cores_d_192": ("bf16", 192, 4, 2, 16, [1, 20, 7], [100, 65, 9], 0),
    "cores_d_256_window": ("f16", 256, 4, 1, 32, [33, 1], [90, 70], 20),
}


def definition(q, kp, vp, table, T, L, scale, window):
    """(o, lse, sum p |v|, sum of the visible |v|) in 64 bits. A row that sees a NaN or an infinite
    score is NaN; one whose scores are all -inf sees nothing."""
    total, Hq, d = q.shape
    Hkv, page = kp.shape[1], kp.shape[2]
    o = torch.full((total, Hq, d), NAN, dtype=torch.float64, device="cuda")
    lse = torch.full((total, Hq), NAN, dtype=torch.float64, device="cuda")
    pv, av = torch.zeros_like(o), torch.zeros_like(o)
    at = 0
    for b, (t, l) in enumerate(zip(T, L)):
        ids = table[b, :-(-l // page)].long()
        j, pos = torch.arange(l, device="cuda"), torch.arange(l - t, l, device="cuda")
        see = (j[None] <= pos[:, None]) & (j[None] > pos[:, None] - (window or l))
        for g in range(Hkv):
            k = kp[ids, g].reshape(-1, d)[:l].double()
            v = vp[ids, g].reshape(-1, d)[:l].double()
            for h in range(g * (Hq // Hkv), (g + 1) * (Hq // Hkv)):
                x = q[at:at + t, h].double()
                s = torch.where(see, x @ k.T * scale, -INF)
                lost = (s.isnan() | (s == INF)).any(1)
                e = torch.logsumexp(torch.where(lost[:, None], -INF, s), 1)
                p = torch.exp(s - torch.where(e == -INF, 0.0, e)[:, None])
                p = torch.where(lost[:, None] | ~see, 0.0, p)
                o[at:at + t, h] = torch.where(lost[:, None], NAN, p @ v)
                lse[at:at + t, h] = torch.where(lost, NAN, e)
                pv[at:at + t, h], av[at:at + t, h] = p @ v.abs(), see.double() @ v.abs()
        at += t
    return o, lse, pv, av


def inputs(name):
    dtype, d, Hq, Hkv, page, T, L, window = CASES[name]
    dtype = DTYPES[dtype]
    kp, vp, table, _ = make_cache(L, Hkv, d, page, dtype, 60 + len(name))
    q = randn((sum(T), Hq, d), dtype, 61 + len(name))
    ld = torch.tensor(L, dtype=torch.int32)
    return [x.cuda() for x in (q, kp, vp, table, cu(T), ld)], T, L, window, d ** -0.5


def check(lib, args, T, L, window, scale):
    o, lse = lib.attn_paged(*args, max_q=max(T), window=window)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
    ro, rl, pv, av = definition(*args[:4], T, L, scale, window)
    lost = rl.isnan()
    assert lost.any()
    assert torch.equal(lse.isnan(), lost)
    assert torch.equal(o.isnan(), lost[..., None].expand_as(o))
    # The others: one rounding of the result, one of each probability (relative, or half the type's
    # smallest step against a sum of at least 1), scores off by (d + 8) 2^-24 sum |q_c k_c| scale < 2^-13, twice.
    half = HALF_STEP[args[0].dtype]
    bound = half * ro.abs() * 1.01 + (half * 1.01 + 2.0 ** -12) * pv + LEAST[args[0].dtype] * (av / 2 + 1)
    assert ((o.double() - ro).abs() <= bound)[~lost].all()
    same = torch.isneginf(lse) & torch.isneginf(rl)  # (their difference is no number)
    assert (same | ((lse.double() - rl).abs() <= 2.0 ** -13 + 2.0 ** -18))[~lost].all()
    again = lib.attn_paged(*args, max_q=max(T), window=window)
    assert torch.equal(torch.nan_to_num(again[0], 5.0), torch.nan_to_num(o, 5.0))
    return o, lse, lost


@pytest.mark.parametrize("name", CASES)
def test_nan_in_a_query_row(lib, name):
    """The row is NaN, in o and lse; every other row has the bits that it had."""
    args, T, L, window, scale = inputs(name)
    clean = lib.attn_paged(*args, max_q=max(T), window=window)
    q = args[0]
    rows = sorted({0, sum(T) // 2, sum(T) - 1})
    for i, r in enumerate(rows):
        q[r, i % q.shape[1], (7 * i) % q.shape[2]] = NAN
    o, lse, lost = check(lib, args, T, L, window, scale)
    assert int(lost.sum()) == len(rows)
    assert torch.equal(o[~lost], clean[0][~lost]) and torch.equal(lse[~lost], clean[1][~lost])


@pytest.mark.parametrize("where", ["early", "middle", "last"])
@pytest.mark.parametrize("name", CASES)
def test_nan_in_a_key(lib, name, where):
    """Every row that sees the key is NaN, in whole and in cut items alike; the others have the bits
    that they had, those behind it in the same tile among them."""
    args, T, L, window, scale = inputs(name)
    clean = lib.attn_paged(*args, max_q=max(T), window=window)
    q, kp, _, table = args[:4]
    page = kp.shape[2]
    for b in {0, len(L) - 1}:
        low = max(0, L[b] - T[b] - window + 1) if window else 0
        j = {"early": low, "middle": (low + L[b]) // 2, "last": L[b] - 1}[where]
        kp[table[b, j // page].long(), 0, j % page, 3] = NAN
    o, lse, lost = check(lib, args, T, L, window, scale)
    assert torch.equal(o[~lost], clean[0][~lost]) and torch.equal(lse[~lost], clean[1][~lost])


@pytest.mark.parametrize("name", CASES)
def test_infinite_scores(lib, name):
    """A key with an infinity: rows whose score it makes +inf are NaN, for rows whose score it makes
    -inf it does not count."""
    args, T, L, window, scale = inputs(name)
    _, kp, _, table = args[:4]
    page = kp.shape[2]
    for b in {0, len(L) - 1}:
        j = max(0, L[b] - T[b] - 3)
        kp[table[b, j // page].long(), 0, j % page, 5] = INF
    check(lib, args, T, L, window, scale)


@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("T", [1, 60])
def test_rows_whose_every_score_is_minus_infinity(lib, d, T):
    """They count as rows without keys: o = 0, lse = -inf, as the sum of the exponentials is 0."""
    L = [700, 60]
    kp, vp, table, _ = make_cache(L, 2, d, 16, torch.bfloat16, 71)
    q = randn((2 * T, 4, d), torch.bfloat16, 72)
    kp[..., 0] = -INF
    q[..., 0] = q[..., 0].abs() + 1.0
    args = [x.cuda() for x in (q, kp, vp, table, cu([T, T]), torch.tensor(L, dtype=torch.int32))]
    o, lse = lib.attn_paged(*args, max_q=T)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("name", ["decode_cut", "decode_whole", "tiles_cut", "tiles_whole", "cores_d_192"])
def test_nan_in_a_value(lib, name):
    """At the last token's own place, which only that token sees with a probability above 0: its
    column of o is NaN, lse and the token's other columns have the bits that they had."""
    args, T, L, window, scale = inputs(name)
    clean = lib.attn_paged(*args, max_q=max(T), window=window)
    vp, table = args[2], args[3]
    page, G = vp.shape[2], args[0].shape[1] // vp.shape[1]
    vp[table[0, (L[0] - 1) // page].long(), 0, (L[0] - 1) % page, 9] = NAN
    o, lse = lib.attn_paged(*args, max_q=max(T), window=window)
    row = T[0] - 1
    assert o[row, :G, 9].isnan().all() and torch.equal(lse, clean[1])
    keep = torch.ones(args[0].shape[2], dtype=torch.bool, device="cuda")
    keep[9] = False
    assert torch.equal(o[row][:, keep], clean[0][row][:, keep])
    assert torch.equal(o[row, G:], clean[0][row, G:]) and torch.equal(o[T[0]:], clean[0][T[0]:])


@pytest.mark.parametrize("G", [2, 8, 32])
@pytest.mark.parametrize("d", [64, 128])
def test_packed_decode_through_the_same_pass(lib, d, G):
    """attn_decode's persistent pass ends its pieces with the same code."""
    lens = [3000, 1, 500]
    kc, vc = (randn((sum(lens) * 2 * d,), torch.bfloat16, 73 + i).cuda() for i in range(2))
    q = randn((3, 2 * G, d), torch.bfloat16, 75).cuda()
    ld = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = lib.attn_decode(q, kc, vc, ld, Hkv=2)
    kc[(1000 * d) + 4] = NAN  # sequence 0, KV head 0, token 1000
    o, lse = lib.attn_decode(q, kc, vc, ld, Hkv=2)
    assert o[0, :G].isnan().all() and lse[0, :G].isnan().all()
    assert torch.equal(o[0, G:], clean[0][0, G:]) and torch.equal(o[1:], clean[0][1:])
    assert torch.equal(lse[1:], clean[1][1:])
