"""The gradient of rope through autograd."""
import numpy as np
import pytest
import torch

import bit_quantized_attention_sage_b200 as sage
import cache_ref as ref
from test_gpu_rope_op import DTS, check

pytestmark = pytest.mark.gpu


def rand(shape, seed, dt="fp32"):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DTS[dt]).cuda()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_of_rope(layout, dt, inverse):
    B, H, N, D, R = 2, 3, 37, 64, 48
    f, amp = sage.rope_freqs(R, scaling=("yarn", 8.0, 100))
    pos = torch.randint(0, 10 ** 6, (B, N), generator=torch.Generator().manual_seed(1))
    x, dy = rand((B, H, N, D), 2, dt), rand((B, H, N, D), 3, dt)
    want = sage.rope(x, pos.cuda(), f, layout, amp, inverse)
    assert want.grad_fn is None
    x.requires_grad_()
    y = sage.rope(x, pos.cuda(), f, layout, amp, inverse)
    assert torch.equal(y, want)
    y.backward(dy)
    # the transposed map of the formula, in 64 bits
    check(dy, x.grad, pos, f.cpu().numpy(), layout, amp, not inverse)
    with torch.no_grad():
        assert sage.rope(x, pos.cuda(), f, layout, amp, inverse).grad_fn is None
    z = sage.rope(x.detach(), pos.cuda(), f, layout, amp, inverse, out=torch.empty_like(x))
    assert z.grad_fn is None and torch.equal(z, want)


def test_gradient_against_differences():
    # rope is linear: a step of 1/8 (exact in fp32) gives the slope up to the
    # rounding of the two results, 2^-22 of |y| each and of the sums
    f, _ = sage.rope_freqs(32)
    pos = torch.arange(9, device="cuda") * 1000
    x, dy = rand((1, 2, 9, 40), 4).requires_grad_(), rand((1, 2, 9, 40), 5)
    y = sage.rope(x, pos, f)
    y.backward(dy)
    for at in ((0, 0, 3, 1), (0, 1, 8, 31), (0, 0, 7, 39)):
        e = torch.zeros_like(x)
        e[at] = 0.125
        step = (sage.rope(x.detach() + e, pos, f).double() - y.detach().double()) * 8
        slope = (step * dy.double()).sum()
        tol = 8 * 2.0 ** -21 * (y.detach().double().abs() * dy.double().abs())[0, at[1], at[2]].sum()
        assert abs(slope - x.grad[at]) <= tol + 1e-6


def test_gradients_of_broadcast_and_expanded():
    # an input broadcast over the heads, a result summed (its gradient an
    # expanded one), and the gradient's gradient
    f, _ = sage.rope_freqs(64)
    pos = torch.arange(5, device="cuda")
    x = rand((1, 1, 5, 64), 6).requires_grad_()
    y = sage.rope(x.expand(2, 4, 5, 64), pos, f, layout="half")
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    one = ref.rope(torch.ones(1, 1, 5, 64), np.arange(5)[None], f.cpu().numpy(), "half", 1.0, True)
    assert np.abs(g.detach().double().cpu().numpy() - 8 * one).max() <= 8 * 24 * 2.0 ** -24
    w = rand((1, 2, 5, 64), 7).requires_grad_()
    v = rand((1, 2, 5, 64), 8).requires_grad_()
    (g,) = torch.autograd.grad((sage.rope(w, pos, f) * v).sum(), w, create_graph=True)
    (h,) = torch.autograd.grad(g.sum(), v)
    assert torch.equal(h, sage.rope(torch.ones_like(w), pos, f).detach())


def test_gradient_on_another_stream():
    f, _ = sage.rope_freqs(64)
    pos = torch.arange(500, device="cuda")
    x, dy = rand((1, 4, 500, 64), 9).requires_grad_(), rand((1, 4, 500, 64), 10)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = sage.rope(x, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    y.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(x.grad, sage.rope(dy, pos, f, inverse=True))


def test_refusals_where_a_gradient_is_recorded():
    f, _ = sage.rope_freqs(64)
    pos = torch.arange(5, device="cuda")
    x = rand((1, 4, 5, 64), 11).requires_grad_()
    with pytest.raises(ValueError):
        sage.rope(x, pos, f, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        sage.rope(x, pos, f.clone().requires_grad_())
    with pytest.raises(ValueError):
        sage.rope(x.detach(), pos, f.clone().requires_grad_())
    p = pos.clone()
    y = sage.rope(x, p, f)
    p.add_(1)  # the backward pass would turn by other angles
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_captured_forward_and_backward():
    # (no eager graph of x may live meanwhile: torch keeps the leaf's node on
    # that graph's stream, for every operator)
    f, _ = sage.rope_freqs(64)
    pos = torch.arange(70, device="cuda")
    x, dy = rand((2, 4, 70, 64), 12, "bf16").requires_grad_(), rand((2, 4, 70, 64), 13, "bf16")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = sage.rope(x, pos, f, layout="half")
        (dx,) = torch.autograd.grad(y, x, dy)
    for seed in (14, 15):
        with torch.no_grad():
            x.copy_(rand(x.shape, seed, "bf16"))
            dy.copy_(rand(x.shape, seed + 9, "bf16"))
        pos.add_(1000)
        g.replay()
        with torch.no_grad():
            assert torch.equal(y, sage.rope(x, pos, f, layout="half"))
            assert torch.equal(dx, sage.rope(dy, pos, f, layout="half", inverse=True))
