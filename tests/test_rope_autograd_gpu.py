"""attn_rope in an autograd graph: its gradient is attn_rope_bwd's, and the formula's."""
import numpy as np
import pytest
import torch

from oracle import paged as ref
from paged_cases import DTYPES, HALF_STEP, LEAST, randn

pytestmark = pytest.mark.gpu


def inputs(lib, dt, d, rot, Hq=6, Hkv=2, N=19, B=2):
    turns, amp = lib.attn_rope_turns(rot, scaling="parts", factor=4)
    pos = torch.arange(300, 300 + N, dtype=torch.int32)
    q, k = randn((B, Hq, N, d), dt, 1).cuda(), randn((B, Hkv, N, d), dt, 2).cuda()
    return q, k, pos, turns, amp


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 128), ("f16", 64, 32), ("f16", 80, 20)])
def test_gradient(lib, dtype, d, rot, interleaved):
    dt = DTYPES[dtype]
    q, k, pos, turns, amp = inputs(lib, dt, d, rot)
    rest = (pos.cuda(), turns.cuda(), amp, interleaved)
    gq, gk = randn(q.shape, dt, 3).cuda(), randn(k.shape, dt, 4).cuda()
    want = lib.attn_rope(q, k, *rest)
    dq, dk = lib.attn_rope_bwd(gq, gk, *rest)
    a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
    y = lib.attn_rope(a, b, *rest)
    assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
    got = torch.autograd.grad(y, (a, b), (gq, gk))
    assert torch.equal(got[0], dq) and torch.equal(got[1], dk)
    # the formula: one rounding, and 2^-21 of the pair for the 32-bit rotation (a pair is at most twice the largest)
    for g, x in zip(got, (gq, gk)):
        w = ref.rope_ref(x.cpu(), pos.numpy(), turns, amp, interleaved, True)
        bound = HALF_STEP[dt] * np.abs(w) * (1 + 2.0 ** -8) + 2 * float(x.abs().max()) * amp * 2.0 ** -21 + LEAST[dt]
        assert (np.abs(g.double().cpu().numpy() - w) <= bound).all()
    # one of them only, through either output
    y = lib.attn_rope(a, k, *rest)
    assert torch.equal(torch.autograd.grad(y[0], a, gq)[0], dq)
    y = lib.attn_rope(q, b, *rest)
    assert torch.equal(torch.autograd.grad(y[1], b, gk)[0], dk)
    y = lib.attn_rope(a, None, *rest)
    assert y[1] is None and torch.equal(torch.autograd.grad(y[0], a, gq)[0], dq)
    assert not lib.attn_rope(q, k, *rest)[0].requires_grad
    with torch.no_grad():
        assert not lib.attn_rope(a, b, *rest)[0].requires_grad


def test_gradient_against_differences(lib):
    """The map is linear, so its difference quotient is exact at any step: sum(g rope(x)) for unit x."""
    turns, amp = lib.attn_rope_turns(16)
    pos, tg = torch.tensor([3, 500], dtype=torch.int32).cuda(), turns.cuda()
    g = randn((1, 1, 2, 24), torch.float16, 4).cuda()
    x = torch.zeros(1, 1, 2, 24, dtype=torch.float16, device="cuda", requires_grad=True)
    (dx,) = torch.autograd.grad(lib.attn_rope(x, None, pos, tg, 1.25)[0], x, g)
    for n in range(2):
        for c in range(24):
            e = torch.zeros_like(x)
            e[0, 0, n, c] = 1.0
            d = float((lib.attn_rope(e, None, pos, tg, 1.25)[0].double() * g.double()).sum())
            # y has two values of at most 1.25, each rounded by 2^-11; dx is rounded once
            size = float(g[0, 0, n].abs().max())
            assert abs(d - float(dx[0, 0, n, c])) <= 2.0 ** -11 * (2 * 1.25 * size + abs(d)) + 1e-6


def test_gradients_of_other_layouts(lib):
    """Gradients that are broadcast, transposed or offset; broadcast and sliced inputs."""
    q, k, pos, turns, amp = inputs(lib, torch.float16, 64, 64)
    rest = (pos.cuda(), turns.cuda(), amp)
    a = q.clone().requires_grad_()
    y, _ = lib.attn_rope(a, None, *rest)
    ones = torch.ones_like(y)
    want, _ = lib.attn_rope_bwd(ones, None, *rest)
    y.sum().backward()  # a gradient of strides 0
    assert torch.equal(a.grad, want)
    wide = torch.ones(2, 6, 19, 67, dtype=torch.float16, device="cuda")[..., 2:66]  # rows not on 16 bytes
    y, _ = lib.attn_rope(a, None, *rest)
    assert torch.equal(torch.autograd.grad(y, a, wide)[0], want)
    y, _ = lib.attn_rope(a, None, *rest)
    turned = torch.ones(2, 6, 64, 19, dtype=torch.float16, device="cuda").transpose(2, 3)
    assert torch.equal(torch.autograd.grad(y, a, turned)[0], want)
    # one head shared by all: its gradient is the sum of theirs
    one = q[:, :1].clone().requires_grad_()
    y, _ = lib.attn_rope(one.expand(2, 6, 19, 64), None, *rest)
    g = randn(q.shape, torch.float16, 5).cuda()
    (got,) = torch.autograd.grad(y, one, g)
    each, _ = lib.attn_rope_bwd(g, None, *rest)
    assert torch.equal(got, each.sum(1, keepdim=True))
    # q and k as parts of one projection
    x = randn((2, 19, 10, 64), torch.float16, 6).cuda().requires_grad_()
    parts = x.transpose(1, 2)
    y = lib.attn_rope(parts[:, :6], parts[:, 6:8], *rest)
    (got,) = torch.autograd.grad((y[0] * 2).sum() + y[1].sum(), x)
    gq, gk = lib.attn_rope_bwd(torch.full_like(y[0], 2.0), torch.ones_like(y[1]), *rest)
    assert torch.equal(got[:, :, :6].transpose(1, 2), gq) and torch.equal(got[:, :, 6:8].transpose(1, 2), gk)
    assert not got[:, :, 8:].any()


def test_second_derivative_and_back(lib):
    """The gradient's own gradient is the rotation again."""
    q, _, pos, turns, amp = inputs(lib, torch.float16, 64, 64)
    rest = (pos.cuda(), turns.cuda(), amp)
    a, g = q.clone().requires_grad_(), randn(q.shape, torch.float16, 7).cuda().requires_grad_()
    (dx,) = torch.autograd.grad(lib.attn_rope(a, None, *rest)[0], a, g, create_graph=True)
    u = randn(q.shape, torch.float16, 8).cuda()
    (dg,) = torch.autograd.grad(dx, g, u)
    assert torch.equal(dg, lib.attn_rope(u, None, *rest)[0])
    y, _ = lib.attn_rope_bwd(a, None, *rest)
    assert torch.equal(torch.autograd.grad(y, a, u)[0], lib.attn_rope(u, None, *rest)[0])


def test_outputs_given_with_a_gradient_are_refused(lib):
    q, k, pos, turns, amp = inputs(lib, torch.bfloat16, 64, 64)
    rest = (pos.cuda(), turns.cuda(), amp)
    a = q.clone().requires_grad_()
    for kw in (dict(q_out=torch.empty_like(q)), dict(k_out=torch.empty_like(k))):
        with pytest.raises(ValueError, match="gradient"):
            lib.attn_rope(a, k, *rest, **kw)
    with pytest.raises(ValueError, match="gradient"):
        lib.attn_rope(q, k, *rest, q_out=a)
    with torch.no_grad():
        lib.attn_rope(a, k, *rest, q_out=a)
    want, _ = lib.attn_rope(q, k, *rest)
    assert torch.equal(a, want)
    with pytest.raises(ValueError):  # what the call refuses otherwise it refuses here
        lib.attn_rope(a.float(), k, *rest)


def test_on_a_given_stream_and_captured(lib):
    q, k, pos, turns, amp = inputs(lib, torch.bfloat16, 128, 128)
    rest = (pos.cuda(), turns.cuda(), amp)
    gq, gk = randn(q.shape, torch.bfloat16, 3).cuda(), randn(k.shape, torch.bfloat16, 4).cuda()
    want = lib.attn_rope(q, k, *rest) + lib.attn_rope_bwd(gq, gk, *rest)
    for side in (torch.cuda.Stream(), torch.cuda.default_stream(), torch.cuda.Stream().cuda_stream):
        a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
        torch.cuda.synchronize()
        y = lib.attn_rope(a, b, *rest, stream=side)
        torch.cuda.synchronize()
        got = y + torch.autograd.grad(y, (a, b), (gq, gk))
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(got, want))
    a, b = q.clone().requires_grad_(), k.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(lib.attn_rope(a, b, *rest), (a, b), (gq, gk))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lib.attn_rope(a, b, *rest)
        got = y + torch.autograd.grad(y, (a, b), (gq, gk))
    for t in got:
        t.detach().zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in zip(got, want))
