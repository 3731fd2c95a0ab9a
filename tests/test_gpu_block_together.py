"""The operators of a regularised block together, as a network uses them: a training step of group norm with
GELU and dropout, the channel mix and dropout into the residual stream, channels first and as tokens; the
step in a captured graph whose replays draw masks of their own; and the trained mix served in 4-bit floats."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import block as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, C, GRID, G = 3, 24, (9, 13), 4
P = GRID[0] * GRID[1]
SEED = 77


def block(x, w, b, A, bias, step):
    prm = fno.GroupNormParams(G, 1e-5, w, b, act=1)
    u = fno.group_norm(x, prm, fno.Dropout(0.2, SEED, 1000, step=step))
    v = fno.channel_mix(u, A, bias, act=0)
    return fno.dropout_residual(v, fno.Dropout(0.5, SEED, 2000, unit="channel", step=step), x)


def leaves():
    rng = np.random.default_rng(3)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().to(DEV).requires_grad_()  # noqa: E731
    return t(B, C, *GRID), t(C), t(C), t(C, C), t(C)


def plain(x, w, b, A, bias, step):
    """The block in float64; the mix keeps its input in 8 bits, whose gradient is that at the kept values."""
    f1 = torch.from_numpy(ref.drop_factor(B, C, P, False, 0.2, SEED, 1000 + step)).to(DEV).view(B, C, *GRID)
    f2 = torch.from_numpy(ref.drop_factor(B, C, P, False, 0.5, SEED, 2000 + step, "channel")).to(DEV).view(B, C, 1, 1)
    h = x.reshape(B, G, -1)
    h = (h - h.mean(-1, keepdim=True)) / torch.sqrt(h.var(-1, unbiased=False, keepdim=True) + 1e-5)
    z = h.reshape(x.shape) * w.view(1, -1, 1, 1) + b.view(1, -1, 1, 1)
    u = z * torch.special.ndtr(z) * f1
    v = torch.einsum("oi,bihw->bohw", A, u) + bias.view(1, -1, 1, 1)
    return x + v * f2


@pytest.mark.parametrize("k", [0, 5])
def test_training_step(k):
    step = torch.full((1,), k, dtype=torch.int64, device=DEV)
    t = leaves()
    y = block(*t, step)
    gy = torch.randn(y.shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    got = torch.autograd.grad(y, t, gy)
    d = [v.detach().double().requires_grad_() for v in t]
    yr = plain(*d, k)
    want = torch.autograd.grad(yr, d, gy.double())
    assert ((y.double() - yr).abs().max() / yr.abs().max()) < 2e-6
    for i, (a, r) in enumerate(zip(got, want)):
        # the weight's gradient takes u from 8 bits: blocks of 32 values off by half of 2^-6 of their largest, at random
        tol = 2.0 ** -7 if i == 3 else 4e-6
        assert ((a.double() - r).norm() / r.norm()) < tol, i


def test_step_in_a_captured_graph():
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    t = leaves()
    gy = torch.randn(B, C, *GRID, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(block(*t, step), t, gy)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = block(*t, step)
        got = torch.autograd.grad(y, t, gy)
    ys = []
    for k in range(3):
        step.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        ys.append(y.detach().clone())
        d = [v.detach().double().requires_grad_() for v in t]
        yr = plain(*d, k)
        assert ((y.double() - yr).abs().max() / yr.abs().max()) < 2e-6
        want = torch.autograd.grad(yr, d, gy.double())
        assert ((got[0].double() - want[0]).norm() / want[0].norm()) < 4e-6
    assert not torch.equal(ys[0], ys[1])


def test_serving_in_four_bits():
    x, w, b, A, bias = (v.detach() for v in leaves())
    with torch.no_grad():
        u = fno.group_norm(x, fno.GroupNormParams(G, 1e-5, w, b, act=1))
        y = fno.channel_mix_mx4(u, fno.Mx4Weight(A), bias, add=x)
    u3, x3 = (t.double().cpu().numpy().reshape(B, C, P) for t in (u, x))
    want, size = ref.mx4_mix(ref.mx4_trip(u3), ref.mx4_trip(A.double().cpu().numpy()), bias.double().cpu().numpy(), x3, 0)
    got = y.double().cpu().numpy().reshape(B, C, P)
    assert (abs(got - want) <= 64 * 2.0 ** -24 * size).all()


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own."""
    a, c = torch.randn(2, 8, 30000, device=DEV), torch.randn(2, 30000, 8, device=DEV)
    prm = [fno.GroupNormParams(2, act=2), fno.GroupNormParams(2, act=1, channels_last=True)]
    want = [fno.group_norm(a, prm[0]), fno.group_norm(c, prm[1])]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for i, t in enumerate((a, c)):
            with torch.cuda.stream(s[i]):
                outs.append((i, fno.group_norm(t, prm[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)
