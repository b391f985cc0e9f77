"""Page operations on rows that have given up pages in front of a sliding window."""
import pytest
import torch

from oracle import paged as ref
from paged_cases import cu, make_cache, randn

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def give_up(table, refs, b, n):
    """Row b's first n pages, as the documentation says."""
    refs[table[b, :n].long()] -= 1
    table[b, :n] = -1


# Few pages go through one kernel, many through the cluster and its copy kernel.
@pytest.mark.parametrize("spare", [40, 30000])
@pytest.mark.parametrize("layers", [None, 2])
def test_update_and_compaction_leave_the_entries(lib, spare, layers):
    lens, page = [70, 3, 100, 33, 64], 16
    kp, vp, table, refs = make_cache(lens, 2, 8, page, torch.bfloat16, 1, spare=spare, width=9, layers=layers)
    give_up(table, refs, 0, 3)
    give_up(table, refs, 2, 5)
    at = 1 if layers else 0
    for source, add in (([0, 1, 2, 3, 4], [1] * 5), ([2, 0, 2, -1, 0], [0, 30, 1, 20, 1]),
                        ([-1, 1, -1, 3, 4], [5, 0, 0, 40, 16])):
        kg, vg = kp.cuda(), vp.cuda()
        t, l, r, info = lib.attn_pages_update(kg, vg, table.cuda(), ints(lens), refs.cuda(), ints(source), ints(add))
        wt, wl, wr, winfo, copies = ref.update_ref(table, lens, refs, source, add, page)
        assert info.tolist() == winfo == [0, 0]
        assert t.tolist() == wt and l.tolist() == wl and r.tolist() == wr
        for a, b in copies:
            for pool in (kp, vp):
                pool.select(at, b).copy_(pool.select(at, a))
        assert torch.equal(kg.cpu(), kp) and torch.equal(vg.cpu(), vp)
        assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
        table, lens, refs = torch.tensor(wt, dtype=torch.int32), wl, torch.tensor(wr, dtype=torch.int32)
        t, r, info = lib.attn_pages_compact(kg, vg, table.cuda(), ints(lens), refs.cuda())
        wt, wr, winfo, moves = ref.compact_ref(table, lens, refs, page)
        assert t.tolist() == wt and r.tolist() == wr and info.tolist() == winfo
        assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
    table[1, 0] = -2  # any other id outside the pool is still an error
    lib.attn_pages_compact(kg, vg, table.cuda(), ints(lens), refs.cuda())
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2001)
    lib.attn_pages_update(kg, vg, table.cuda(), ints(lens), refs.cuda(), ints([0, 1, 2, 3, 4]), ints([0] * 5))
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2001)


def test_decoding_under_a_window_in_a_pool_that_holds_little_more_than_it(lib):
    """Steps of one token: grow, append, attend under the window, give up what it has left behind.
    The pages run out unless they go round; the results are those of a cache that keeps all."""
    B, Hq, Hkv, d, page, window, steps = 3, 8, 2, 64, 16, 40, 120
    width = 12
    per_row = -(-window // page) + 2
    P = B * per_row
    pools = [torch.full((n, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
             for n in (P, P, B * width, B * width)]
    turns = lib.attn_rope_turns(d)[0].cuda()
    c, same, one = cu([1] * B).cuda(), ints(list(range(B))), ints([1] * B)
    small = [torch.full((B, width), -1, dtype=torch.int32, device="cuda"), ints([0] * B), ints([0] * P)]
    large = [small[0].clone(), ints([0] * B), ints([0] * (B * width))]
    g = torch.Generator().manual_seed(3)
    for step in range(steps):
        x = torch.randn((B, Hq + 2 * Hkv, d), generator=g).to(torch.bfloat16).cuda()
        out = []
        for (kp, vp), st in ((pools[:2], small), (pools[2:], large)):
            st[0], st[1], st[2], info = lib.attn_pages_update(kp, vp, *st, same, one)
            assert info.tolist() == [0, 0], step
            q = lib.attn_rope_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kp, vp, st[0], c, st[1], turns)
            out.append(lib.attn_paged(q, kp, vp, st[0], c, st[1], max_q=1, window=window))
        assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
        L = int(small[1][0])
        n = max(0, L + 1 - window) // page  # pages that the next token does not see either
        gone = small[0][:, :n]
        small[2].index_add_(0, gone[gone >= 0].long(), torch.full_like(gone[gone >= 0], -1))
        gone.fill_(-1)
    assert L == steps and int((small[2] > 0).sum()) <= P
