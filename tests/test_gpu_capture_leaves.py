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


@pytest.mark.parametrize("op", ["mix", "norm", "group norm", "dropout"])
def test_streams_that_joined_the_capture(op):
    """Two calls of the same leaves on two streams of one capture, the accumulators of the first's."""
    leaves, call, _ = _case(op)
    first = call()
    gy, gz = torch.randn_like(first), torch.randn_like(first)
    del first
    want = torch.autograd.grad((call(), call()), leaves, (gy, gz))
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        y = call()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z = call()
        main.wait_stream(side)
        got = torch.autograd.grad((y, z), leaves, (gy, gz))
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        for a, r in zip(got, want):
            # two terms, added in either order
            assert (a - r).abs().max() <= 2.0 ** -23 * r.abs().max()


@pytest.mark.parametrize("op", ["mix", "group norm"])
def test_another_stream_than_the_default(op):
    """An eager graph on a stream of its own, which has not joined the capture."""
    leaves, call, _ = _case(op)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        eager = call()
    torch.cuda.synchronize()
    gy = torch.ones_like(eager)
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            torch.autograd.grad(call(), leaves, gy)
    assert torch.isfinite(eager).all()
