"""What the paged operators write in place, autograd's check of saved tensors sees."""
import pytest
import torch

from paged_cases import cu, make_cache, randn

pytestmark = pytest.mark.gpu


def test_versions_move_with_what_is_written(lib):
    kp, vp, table, refs = (x.cuda() for x in make_cache([20, 5], 2, 64, 16, torch.bfloat16, 1))
    lens = torch.tensor([20, 5], dtype=torch.int32).cuda()
    c, turns = cu([3, 1]).cuda(), lib.attn_rope_turns(64)[0].cuda()
    x = randn((4, 8, 64), torch.bfloat16, 2).cuda()
    q, k, v = x[:, :4].contiguous(), x[:, 4:6].contiguous(), x[:, 6:].contiguous()
    o, lse = torch.empty_like(q), torch.empty(4, 4, device="cuda")
    source, add = torch.arange(2, dtype=torch.int32).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    outs = dict(table_out=torch.empty_like(table), lens_out=torch.empty_like(lens), refs_out=torch.empty_like(refs),
                info=torch.empty(2, dtype=torch.int32, device="cuda"))
    every = [kp, vp, table, refs, lens, c, turns, q, k, v, o, lse, source, add, *outs.values()]

    def moved(call, *written):
        before = [t._version for t in every]
        call()
        for t, n in zip(every, before):
            assert t._version == n + any(t is w for w in written)

    moved(lambda: lib.attn_paged(q, kp, vp, table, c, lens))
    moved(lambda: lib.attn_paged(q, kp, vp, table, c, lens, o=o, lse=lse), o, lse)
    moved(lambda: lib.attn_rope_append(q, k, v, kp, vp, table, c, lens, turns), kp, vp)
    moved(lambda: lib.attn_rope_append(q, k, v, kp, vp, table, c, lens, turns, q_out=q), kp, vp, q)
    pos = torch.arange(4, dtype=torch.int32).cuda()
    four = [t[None].transpose(1, 2) for t in (q, k, o)]  # (views share their base's version)
    moved(lambda: lib.attn_rope(four[0], four[1], pos, turns))
    moved(lambda: lib.attn_rope(four[0], four[1], pos, turns, q_out=four[0], k_out=four[1]), q, k)
    moved(lambda: lib.attn_rope_bwd(four[0], None, pos, turns, dq_in=four[2]), o)
    moved(lambda: lib.attn_pages_update(kp, vp, table, lens, refs, source, add, **outs), kp, vp, *outs.values())
    some = dict(table_out=outs["table_out"], info=outs["info"])
    moved(lambda: lib.attn_pages_compact(kp, vp, table, lens, refs, **some), kp, vp, *some.values())
    with pytest.raises(lib.AttnError):  # a refused call wrote nothing
        moved(lambda: lib.attn_pages_compact(kp, vp, table, lens, refs, table_out=table))


def test_a_graph_that_saved_a_pool_finds_out(lib):
    kp, vp, table, _ = (x.cuda() for x in make_cache([20], 2, 64, 16, torch.bfloat16, 1))
    lens, c, turns = torch.tensor([20], dtype=torch.int32).cuda(), cu([1]).cuda(), torch.zeros(0).double().cuda()
    x = randn((1, 2, 64), torch.bfloat16, 2).cuda()
    w = torch.ones_like(kp, requires_grad=True)
    loss = (w * kp).sum()
    lib.attn_rope_append(x, x, x, kp, vp, table, c, lens, turns)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_inference_tensors(lib):
    with torch.inference_mode():
        kp, vp, table, _ = (x.cuda() for x in make_cache([20], 2, 64, 16, torch.bfloat16, 1))
        lens, c, turns = torch.tensor([20], dtype=torch.int32).cuda(), cu([1]).cuda(), torch.zeros(0).double().cuda()
        x = randn((1, 2, 64), torch.bfloat16, 2).cuda()
        lib.attn_rope_append(x, x, x, kp, vp, table, c, lens, turns)
        o = torch.empty_like(x)
        lib.attn_paged(x, kp, vp, table, c, lens, o=o)
    lib.attn_paged(x, kp, vp, table, c, lens, o=o)  # and outside of it
    assert torch.isfinite(o.float()).all()
