"""Sliding windows over a paged cache: what lies in front of every token's window is not needed."""
import pytest
import torch

from paged_cases import DTYPES, cu, make_cache, randn

pytestmark = pytest.mark.gpu

NAN = float("nan")

# dtype, d, Hq, Hkv, page, new tokens, cached tokens, window
CASES = {
    "decode": ("bf16", 128, 8, 2, 16, [1, 1, 1, 1], [900, 129, 100, 5000], 100),
    "decode_d64_page_64": ("f16", 64, 8, 4, 64, [1] * 5, [900, 129, 100, 64, 5000], 70),
    "decode_page_8": ("bf16", 128, 32, 1, 8, [1, 1], [1001, 300], 129),
    "decode_page_256": ("bf16", 128, 8, 2, 256, [1, 1], [1001, 3000], 300),
    "decode_many": ("bf16", 128, 8, 2, 16, [1] * 100, [150 + 7 * i for i in range(100)], 77),
    "decode_plan_kernel": ("bf16", 128, 4, 1, 16, [1] * 1200, [60 + i % 300 for i in range(1200)], 50),
    "few_tokens": ("bf16", 128, 16, 4, 16, [4, 7, 8], [900, 333, 2000], 41),
    "window_of_one": ("f16", 64, 8, 2, 16, [1, 1], [401, 129], 1),
    "tiles": ("bf16", 128, 8, 2, 16, [200, 64, 1], [1000, 64, 700], 130),
    "tiles_d64": ("f16", 64, 14, 2, 32, [133, 40, 65], [4000, 900, 1111], 401),
    "tiles_page_128": ("bf16", 128, 8, 2, 128, [200, 90], [3000, 1000], 333),
    "tiles_page_512": ("f16", 128, 8, 2, 512, [200, 90], [3000, 1700], 99),
    "tiles_beyond_l2": ("bf16", 128, 8, 8, 64, [300, 300], [20011, 5000], 3001),
    "one_tile_many": ("bf16", 64, 8, 2, 16, [20] * 80, [300 + 11 * i for i in range(80)], 150),
    "cores_d_192": ("bf16", 192, 4, 2, 16, [1, 20, 7], [700, 365, 90], 45),
    "cores_d_256": ("f16", 256, 4, 1, 32, [33, 1], [290, 470], 20),
}


@pytest.mark.parametrize("what", ["given_up", "nan_pages", "nan_rows"])
@pytest.mark.parametrize("name", CASES)
def test_in_front_of_the_window(lib, name, what):
    """Table entries of -1 for pages wholly in front of every token's window (no error, the same
    bits), and NaN in such pages and in the rows of the window's first page in front of it."""
    dtype, d, Hq, Hkv, page, T, L, window = CASES[name]
    dtype = DTYPES[dtype]
    kp, vp, table, _ = make_cache(L, Hkv, d, page, dtype, 80 + len(name))
    q = randn((sum(T), Hq, d), dtype, 81 + len(name)).cuda()
    c, ld = cu(T).cuda(), torch.tensor(L, dtype=torch.int32).cuda()
    args = dict(max_q=max(T), window=window)
    o, lse = lib.attn_paged(q, kp.cuda(), vp.cuda(), table.cuda(), c, ld, **args)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
    assert o.isfinite().all() and lse.isfinite().all()
    some = False
    for b, (t, l) in enumerate(zip(T, L)):
        first = max(0, l - t - window + 1)  # the first key that any token of the sequence sees
        n = first // page
        some = some or (first > 0 if what == "nan_rows" else n > 0)
        if what == "given_up":
            table[b, :n] = -1
        elif what == "nan_pages":
            kp[table[b, :n].long()], vp[table[b, :n].long()] = NAN, NAN
        else:
            for j in range(0, n + 1):
                to = page if j < n else first % page
                kp[table[b, j].long(), :, :to], vp[table[b, j].long(), :, :to] = NAN, NAN
    assert some
    o2, lse2 = lib.attn_paged(q, kp.cuda(), vp.cuda(), table.cuda(), c, ld, **args)
    assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("T", [1, 50])
def test_a_missing_page_in_the_window_is_reported(lib, d, T):
    """One page further, and a token needs it: reported, at every kind of kernel."""
    L, window, page = [900, 500], 100, 16
    kp, vp, table, _ = make_cache(L, 2, d, page, torch.bfloat16, 91)
    q = randn((2 * T, 8, d), torch.bfloat16, 92).cuda()
    c, ld = cu([T, T]).cuda(), torch.tensor(L, dtype=torch.int32).cuda()
    n = (L[0] - T - window + 1) // page
    for k, want in ((n, lib.ATTN_OK), (n + 1, lib.ATTN_ERR_PAGES)):
        t = table.clone()
        t[0, :k] = -1
        lib.attn_paged(q, kp.cuda(), vp.cuda(), t.cuda(), c, ld, max_q=T, window=window)
        assert lib.attn_get_device_status()[0] == want
