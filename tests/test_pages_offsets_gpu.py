"""Pages whose places lie beyond 32-bit offsets are moved and copied."""
import pytest
import torch

from oracle import paged as ref

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("P", [14, 30000])
def test_pages_move_and_are_copied_beyond_32_bits(lib, P):
    """At least one page moves from, and one is copied from, an element offset above 2^32."""
    lens, page, Hkv, d = [40, 100, 9], 16, 2, 8
    n = Hkv * page * d
    wide = (1 << 32) // (P - 2) // 8 * 8 + 8  # values between pages: page P - 2 lies behind 2^32
    assert (P - 2) * wide > 1 << 32
    big = torch.empty((P - 1) * wide + 2 * n, dtype=torch.bfloat16, device="cuda")
    view = lambda off: big.as_strided((P, Hkv, page, d), (wide, page * d, d, 1), off)  # noqa: E731
    kg, vg = view(0), view(n)
    g = torch.Generator().manual_seed(3)
    kp, vp = (torch.randn((P, Hkv, page, d), generator=g).to(torch.bfloat16) for _ in range(2))
    kg.copy_(kp)
    vg.copy_(vp)
    table = torch.full((3, 9), -1, dtype=torch.int32)
    table[0, :3] = torch.tensor([P - 2, 0, P - 1])  # its last, partly filled page is the last of the pool
    table[1, :7] = torch.tensor([2, 4, 3, 6, 8, 7, 5])
    table[2, :1] = 9
    refs = torch.zeros(P, dtype=torch.int32)
    refs[table[table >= 0].long()] = 1
    t, l, r, info = lib.attn_pages_update(kg, vg, table.cuda(), ints(lens), refs.cuda(), ints([0, 1, 0]), ints([1, 1, 1]))
    wt, wl, wr, winfo, copies = ref.update_ref(table, lens, refs, [0, 1, 0], [1, 1, 1], page)
    assert any(a * wide > 1 << 32 for a, _ in copies)
    assert t.tolist() == wt and l.tolist() == wl and r.tolist() == wr and info.tolist() == winfo == [0, 0]
    t, r, info = lib.attn_pages_compact(kg, vg, t, l, r)
    wt, wr, winfo, moves = ref.compact_ref(wt, wl, wr, page)
    assert int(info[1]) == len(moves) >= 1 and any(a * wide > 1 << 32 for a, _ in moves)
    assert t.tolist() == wt and r.tolist() == wr and info.tolist() == winfo
    for a, b in copies + moves:
        kp[b], vp[b] = kp[a], vp[a]
    assert torch.equal(kg.cpu(), kp) and torch.equal(vg.cpu(), vp)
    assert lib.attn_get_device_status()[0] == lib.ATTN_OK
