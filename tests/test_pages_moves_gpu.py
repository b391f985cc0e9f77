"""Where compaction puts the pages that no row holds."""
import pytest
import torch

from paged_cases import make_cache

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("spare", [60, 30000])  # one kernel, and the cluster with its copy kernel
def test_a_holder_from_outside_finds_its_pages(lib, spare):
    """By the documented rule, from the counts before; or by a row of its own in the table."""
    lens, page = [100, 33, 0, 50], 16
    kp, vp, table, refs = make_cache(lens, 2, 8, page, torch.bfloat16, 2, spare=spare, layers=2)
    free = (refs == 0).nonzero().flatten().tolist()
    pinned = [free[-1], free[len(free) // 2], free[0]]
    refs[pinned] += 1
    own = table[3, :4].tolist()  # row 3 is such a holder's: its four pages follow in the table
    kg, vg = kp.cuda(), vp.cuda()
    t, r, info = lib.attn_pages_compact(kg, vg, table.cuda(), ints(lens), refs.cuda())
    n = int((refs > 0).sum())
    at = torch.arange(len(refs))
    of, to = at[(refs > 0) & (at >= n)], at[(refs <= 0) & (at < n)]
    assert info.tolist() == [n, len(of)] and len(of) >= 2
    now = at.scatter(0, of, to)[pinned]
    assert (now < n).all() and any(int(now[i]) != p for i, p in enumerate(pinned))
    for pool, was in ((kg, kp), (vg, vp)):
        assert torch.equal(pool[:, now.cuda()].cpu(), was[:, pinned])
        assert torch.equal(pool[:, t[3, :4].long()].cpu(), was[:, own])
    assert (r[now.cuda()] == 1).all()
