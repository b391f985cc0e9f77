"""The paged operators on a stream given by argument, with outputs that the call allocates."""
import pytest
import torch

from paged_cases import cu, make_cache, randn

pytestmark = pytest.mark.gpu


def setup(lib, op):
    """(call with a stream, shapes and types of the outputs that it allocates)"""
    T, L, Hq, Hkv, d = [200, 300], [4000, 300], 8, 2, 64
    kp, vp, table, refs = make_cache(L, Hkv, d, 64, torch.bfloat16, 51, spare=40)
    x = randn((500, Hq + 2 * Hkv, d), torch.bfloat16, 52).cuda()
    kp, vp, table, refs, c = kp.cuda(), vp.cuda(), table.cuda(), refs.cuda(), cu(T).cuda()
    lens = torch.tensor(L, dtype=torch.int32).cuda()
    turns = lib.attn_rope_turns(d)[0].cuda()
    q, k, v = x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    i32, b16 = torch.int32, torch.bfloat16
    if op == "paged":
        return (lambda s: lib.attn_paged(q, kp, vp, table, c, lens, stream=s),
                [((500, Hq, d), b16), ((500, Hq), torch.float32)])
    if op == "rope":
        q4, k4 = q[None].transpose(1, 2).contiguous(), k[None].transpose(1, 2).contiguous()
        pos = torch.arange(500, dtype=i32).cuda()
        return (lambda s: lib.attn_rope(q4, k4, pos, turns, stream=s), [(q4.shape, b16), (k4.shape, b16)])
    if op == "append":
        return (lambda s: (lib.attn_rope_append(q, k, v, kp, vp, table, c, lens, turns, stream=s),),
                [((500, Hq, d), b16)])
    same, one = torch.arange(2, dtype=i32).cuda(), torch.ones(2, dtype=i32).cuda()
    if op == "update":
        return (lambda s: lib.attn_pages_update(kp, vp, table, lens, refs, same, one, stream=s),
                [(table.shape, i32), (lens.shape, i32), (refs.shape, i32), ((2,), i32)])
    return (lambda s: lib.attn_pages_compact(kp, vp, table, lens, refs, stream=s),
            [(table.shape, i32), (refs.shape, i32), ((2,), i32)])


@pytest.mark.parametrize("op", ["paged", "rope", "append", "update", "compact"])
def test_outputs_are_not_what_the_current_stream_still_uses(lib, op):
    """Tensors of the outputs' sizes are dropped while work queued on the current stream has yet to
    read them; the given stream does not wait for that work, so the outputs must lie elsewhere."""
    call, shapes = setup(lib, op)
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    held = [torch.full(s, 3, dtype=t, device="cuda") for s, t in shapes]
    seen = [torch.zeros(s, dtype=t, device="cuda") for s, t in shapes]
    where = {t.data_ptr() for t in held}
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # some 0.1 s of the current stream
    for a, b in zip(seen, held):
        a.copy_(b)
    del held, b
    out = call(side)
    assert not any(t.data_ptr() in where for t in out)
    side.synchronize()
    want = [t.clone() for t in out]
    torch.cuda.synchronize()
    assert all((t == 3).all() for t in seen)
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["paged", "rope"])
def test_outputs_used_on_the_current_stream_keep_their_memory(lib, op):
    """Dropped while the current stream, made to wait for the given one, still has to read them."""
    call, _ = setup(lib, op)
    side = torch.cuda.Stream()
    want = call(side)[0]
    torch.cuda.synchronize()
    out = call(side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    got = torch.empty_like(want)
    got.copy_(out)
    del out
    later = [call(side) for _ in range(20)]  # would take its place
    with torch.cuda.stream(side):
        for o in later:
            o[0].zero_()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_the_same_results_and_the_current_stream_as_it_was(lib):
    for op in ("paged", "rope"):
        call, _ = setup(lib, op)
        want = call(None)
        torch.cuda.synchronize()
        side, here = torch.cuda.Stream(), torch.cuda.current_stream()
        out = [call(s) for s in (side, side.cuda_stream, here, here.cuda_stream)]
        assert torch.cuda.current_stream() == here
        torch.cuda.synchronize()
        for got in out:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("op", ["paged", "rope", "append", "update", "compact"])
def test_captured_with_the_stream_given(lib, op):
    """In a capture, with the capturing stream given by argument or not: the graph's own memory."""
    call, _ = setup(lib, op)
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(torch.cuda.current_stream()) + call(None)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want + want))
