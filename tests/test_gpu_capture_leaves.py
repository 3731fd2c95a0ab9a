"""A backward captured into a graph while an eager graph on another stream holds the same leaves is refused, not the end of
the process, for every differentiable function; once that graph is gone the step can be captured."""

import pytest
import torch

import spectral_convolution_amd as fno

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _leaf(*shape):
    return torch.randn(shape, device=DEV, requires_grad=True)


def _case(op):
    """(leaves, the call, what keeps its plan)."""
    x, w, b = _leaf(2, 8, 40), _leaf(8), _leaf(8)
    if op == "mix":
        A, bias, add = _leaf(8, 8), _leaf(8), _leaf(2, 8, 40)
        return (x, A, bias, add), lambda: fno.channel_mix(x, A, bias, add, act=1), None
    if op == "norm":
        v = _leaf(2, 8, 40)
        prm = fno.NormParams("layer", 1e-5, w_post=w, b_post=b)
        return (x, v, w, b), lambda: fno.norm_residual(x, v, prm)[0], None
    if op == "spectral":
        plan = fno.fno_plan_create(2, 2, 4, 4, (16, 16), (4, 4), "f32", 0)
        f, re, im = _leaf(2, 4, 16, 16), _leaf(*plan.split_shape()), _leaf(*plan.split_shape())
        return (f, re, im), lambda: fno.spectral_conv(plan, f, re, im), plan
    if op == "group norm":
        prm = fno.GroupNormParams(2, 1e-5, w, b, act=1)
        return (x, w, b), lambda: fno.group_norm(x, prm), None
    v = _leaf(2, 8, 40)
    return (x, v), lambda: fno.dropout_residual(v, fno.Dropout(0.5, 1), x), None


@pytest.mark.parametrize("op", ["mix", "norm", "spectral", "group norm", "dropout"])
def test_captured_backward(op):
    leaves, call, plan = _case(op)
    try:
        eager = call()
        gy = torch.randn_like(eager)
        want = torch.autograd.grad(call(), leaves, gy)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            y = call()  # its forward eager, its leaves' accumulators of the stream before
        torch.cuda.synchronize()
        with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
                torch.autograd.grad(y, leaves, gy)
        with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
                torch.autograd.grad(call(), leaves, gy)
        del y, eager
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            got = torch.autograd.grad(call(), leaves, gy)
        for _ in range(3):
            for t in got:
                if t.data_ptr() != gy.data_ptr():  # a residual stream's gradient is gy itself
                    t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, r) for a, r in zip(got, want))
    finally:
        fno.fno_plan_destroy(plan)


@pytest.mark.parametrize("op", ["mix", "norm", "spectral"])
def test_captured_forward(op):
    """A forward alone is captured beside the eager graph."""
    leaves, call, plan = _case(op)
    try:
        eager = call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = call()
        for _ in range(3):
            y.detach().zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, eager)
    finally:
        fno.fno_plan_destroy(plan)


@pytest.mark.parametrize("op", ["group norm", "dropout"])
def test_captured_forward_without_gradients(op):
    """Where no backward is wanted the call is captured under torch.no_grad()."""
    leaves, call, _ = _case(op)
    eager = call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(g):
        y = call()
    for _ in range(3):
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager)
