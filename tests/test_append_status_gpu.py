"""attn_rope_append reports bad row offsets and lengths, as attn_paged does."""
import pytest
import torch

from paged_cases import cu, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rot", [64, 20])
@pytest.mark.parametrize("offsets,lens,raw", [
    ([0, 3, 1, 4], [40, 50, 60], 0x2003),   # decreasing
    ([0, 1, 2, 9], [40, 50, 60], 0x2003),   # beyond the packed rows
    ([-2, 1, 2, 4], [40, 50, 60], 0x2003),  # before them
    ([0, 1, 1, 4], [40, 1 << 20, 60], 0x2002),  # a length beyond the table, without new tokens
    ([0, 1, 1, 4], [40, 50, 60], None)])
def test_reported(lib, offsets, lens, raw, rot):
    kp, vp, table, _ = make_cache([40, 50, 60], 2, 64, 16, torch.bfloat16, 9)
    x = randn((4, 6, 64), torch.bfloat16, 10).cuda()
    turns = lib.attn_rope_turns(rot)[0].cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    lib.attn_rope_append(x[:, :2], x[:, 2:4], x[:, 4:], kp.cuda(), vp.cuda(), table.cuda(), i32(offsets), i32(lens),
                         turns)
    assert lib.attn_get_device_status() == ((lib.ATTN_OK, 0) if raw is None else (lib.ATTN_ERR_PAGES, raw))


@pytest.mark.parametrize("at", [0, 300, 2998, 2999])
def test_reported_wherever_in_a_large_batch(lib, at):
    """More sequences than the launch has threads for at once, few tokens."""
    B = 3000
    kp, vp, table, _ = make_cache([5] * 4, 1, 8, 8, torch.float16, 3)
    table = table[:1].expand(B, -1).contiguous()
    x = randn((3, 1, 8), torch.float16, 4).cuda()
    lens = torch.zeros(B, dtype=torch.int32)
    c = cu([0] * (B - 1) + [0])
    turns = torch.zeros(0, dtype=torch.float64).cuda()
    args = (x, x, x, kp.cuda(), vp.cuda(), table.cuda(), c.cuda())
    lib.attn_rope_append(*args, lens.cuda(), turns)
    assert lib.attn_get_device_status() == (lib.ATTN_OK, 0)
    lens[at] = 1 << 20
    lib.attn_rope_append(*args, lens.cuda(), turns)
    assert lib.attn_get_device_status() == (lib.ATTN_ERR_PAGES, 0x2002)
