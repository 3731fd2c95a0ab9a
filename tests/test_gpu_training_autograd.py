"""The training operators as differentiable functions (channel_mix, norm_residual)
against their float64 definitions, the calls behind them replayed from captured
graphs, and the example that trains a network of them.

Gradients are those at the values read back from 8 bits, so the inputs here are such
values already and the oracle's gradients at the inputs are the ones to meet."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import training as ref
from test_gpu_training import ACT
from training_util import DT, LOW, NORM_NAMES, close, norm_case, stored

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]
DEV = "cuda:0"


def kept(pair, dtype):
    """The values an 8-bit checkpoint of a field keeps, as (tensor, float64)."""
    r = ref.round_trip(pair[1], LOW[dtype])
    return torch.from_numpy(r).to(DT[dtype]), r


def leaf(t):
    return t.to(DEV).requires_grad_()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act,bias,add", [(1, True, True), (1, False, True), (0, True, True), (1, True, False)])
@pytest.mark.parametrize("shape", [(2, 5, 7, (33,)), (3, 24, 40, (9, 11)), (1, 64, 64, (3, 5, 7))], ids=str)
def test_channel_mix(dtype, act, bias, add, shape):
    B, I, O, grid = shape
    P = int(np.prod(grid))
    rng = np.random.default_rng(P)
    x = kept(stored(rng, (B, I, P), dtype, spread=True), dtype)
    a = kept(stored(rng, (B, O, P), dtype, spread=True), dtype) if add else None
    A, b = stored(rng, (O, I), dtype, I ** -0.5), stored(rng, (O,), dtype, 0.3)
    gy = stored(rng, (B, O, P), dtype, 0.5)
    tx, tA, tb = leaf(x[0].view(B, I, *grid)), leaf(A[0]), leaf(b[0]) if bias else None
    ta = leaf(a[0].view(B, O, *grid)) if add else None
    y = fno.channel_mix(tx, tA, tb, ta, act)
    assert y.shape == (B, O) + grid
    y.backward(gy[0].to(DEV).view(y.shape))
    b64, a64 = b[1] if bias else 0 * b[1], a[1] if add else None
    (gx, gA, gb, gz), _ = ref.channel_mix_backward(x[1], A[1], b64, a64, gy[1], act)
    zs = ref.mix_pre(abs(x[1]), abs(A[1]), abs(b64), None) + (abs(a64) if add else 0) + 1
    gzs = abs(gy[1]) * (zs if act else 1.0)
    flat = lambda t: t.reshape(t.shape[0], t.shape[1], -1)  # noqa: E731
    close("y", flat(y), ref.channel_mix(x[1], A[1], b64, a64, act), dtype, extra=ACT[dtype], size=zs)
    close("gx", flat(tx.grad), gx, dtype, extra=ACT[dtype], size=np.einsum("oi,bop->bip", abs(A[1]), gzs))
    close("gA", tA.grad, gA, dtype, extra=ACT[dtype], size=np.einsum("bop,bip->oi", gzs, abs(x[1])))
    if bias:
        close("gbias", tb.grad, gb, dtype, extra=ACT[dtype], size=gzs.sum((0, 2)))
    if add:
        close("gadd", flat(ta.grad), gz, dtype, extra=ACT[dtype], size=gzs)


def test_channel_mix_of_strided_and_shifted_inputs():
    """A transposed view, a view off the 16-byte grid and an expanded gradient give what their copies give."""
    rng = np.random.default_rng(4)
    x = stored(rng, (2, 37, 6), "f32")[0].to(DEV).transpose(1, 2)
    add = torch.cat([torch.zeros(1), stored(rng, (2 * 5 * 37,), "f32")[0]]).to(DEV)[1:].view(2, 5, 37)
    A = stored(rng, (6, 5), "f32")[0].to(DEV).t()
    assert not x.is_contiguous() and add.data_ptr() % 16 and not A.is_contiguous()
    got = []
    for f in (lambda t: t.detach().requires_grad_(), lambda t: t.detach().contiguous().clone().requires_grad_()):
        leaves = [f(t) for t in (x, A, add)]
        y = fno.channel_mix(leaves[0], leaves[1], None, leaves[2], 1)
        got.append([y] + list(torch.autograd.grad(y.sum(), leaves)))
    for s, t in zip(*got):
        assert torch.equal(s, t)


def test_channel_mix_gives_only_the_gradients_asked_for():
    rng = np.random.default_rng(5)
    x, A = stored(rng, (2, 8, 40), "f16")[0].to(DEV), stored(rng, (8, 8), "f16")[0].to(DEV)
    assert not fno.channel_mix(x, A).requires_grad
    y = fno.channel_mix(x, A.clone().requires_grad_(), act=1)
    y.sum().backward()
    w = A.clone().requires_grad_()
    (g,) = torch.autograd.grad(fno.channel_mix(x, w, act=1).sum(), w)
    both = [x.clone().requires_grad_(), A.clone().requires_grad_()]
    gx, gA = torch.autograd.grad(fno.channel_mix(*both, act=1).sum(), both)
    assert torch.equal(g, gA) and gx.shape == x.shape


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("keep", ["8bit", "whole"])
@pytest.mark.parametrize("P", [None, 77])
@pytest.mark.parametrize("through", ["y and u", "y", "u"])
def test_norm_residual(dtype, kind, keep, P, through):
    c, prm = norm_case(dtype, 3, 40, P, seed=21)
    for k in ("x", "v"):
        c[k] = kept(c[k], dtype)
    x, v = leaf(c["x"][0]), leaf(c["v"][0])
    p = {k: leaf(t[0]) for k, t in prm.items()}
    y, u = fno.norm_residual(x, v, fno.NormParams(kind, 1e-5, **p), keep=keep)
    out, grads = [], []
    for k, t, g in (("y", y, "gy"), ("u", u, "gu")):
        if k in through.split():
            out.append(t)
            grads.append(c[g][0].to(DEV))
    torch.autograd.backward(out, grads)
    gy = c["gy"][1] if "y" in through.split() else np.zeros_like(c["gy"][1])
    gu = c["gu"][1] if "u" in through.split() else None
    p64 = {k: t[1] for k, t in prm.items()}
    g = ref.norm_residual_backward(p64, kind, 1e-5, c["x"][1], c["v"][1], gy, gu)
    top = lambda t: float(np.max(abs(t).max(1) / (np.std(t, axis=1) + 1e-5 ** 0.5)))  # noqa: E731
    yr, _ = ref.norm_residual(p64, kind, 1e-5, c["x"][1], c["v"][1])
    extra = 8 * 2.0 ** -24 * (top(c["v"][1]) + top(yr)) if kind == "layer" else 16 * 2.0 ** -24
    rms = lambda t: np.sqrt(np.mean(t ** 2))  # noqa: E731
    for k, t in (("gx", x), ("gv", v)):
        close(k, t.grad, g[k][0], dtype, size=np.maximum(g[k][1], rms(g[k][0])), extra=extra)
    for k, t in p.items():
        if gu is None and k.endswith("_pre"):
            assert t.grad is None
        else:
            close("g_" + k, t.grad, g[k][0], dtype, size=g[k][1] + abs(g[k][0]), extra=extra)


def test_norm_residual_of_a_gate_shared_by_the_samples():
    """The gradient of a broadcast gate is the sum over the samples."""
    c, prm = norm_case("f32", 4, 24, 50, seed=22)
    x, v = (c[k][0].to(DEV) for k in ("x", "v"))
    p = {k: t[0].to(DEV) for k, t in prm.items() if k != "gate"}
    one = prm["gate"][0][0].to(DEV).requires_grad_()
    each = one.detach().expand(4, -1).contiguous().requires_grad_()
    for gate in (one.expand(4, -1), each):
        y, u = fno.norm_residual(x, v, fno.NormParams("rms", 1e-5, gate=gate, **p))
        (y.square().sum() + u.sum()).backward()
    close("gate", one.grad, each.grad.double().sum(0).cpu().numpy(), "f32")


def test_norm_residual_without_u():
    c, prm = norm_case("bf16", 2, 24, 50, seed=23)
    p = {k: leaf(t[0]) for k, t in prm.items()}
    x, v = leaf(c["x"][0]), leaf(c["v"][0])
    y, u = fno.norm_residual(x, v, fno.NormParams("rms", 1e-5, **p), with_u=False)
    assert u is None
    y.sum().backward()
    y2, _ = fno.norm_residual(x, v, fno.NormParams("rms", 1e-5, **p))
    assert torch.equal(y, y2) and p["w_pre"].grad is None and p["gate"].grad is not None
    assert torch.equal(x.grad, torch.ones_like(x))


def test_shapes_that_do_not_fit_are_refused():
    x, A = torch.zeros(2, 3, 5, device=DEV), torch.zeros(4, 3, device=DEV)
    with pytest.raises(ValueError, match="A shape"):
        fno.channel_mix(x, torch.zeros(4, 5, device=DEV))
    with pytest.raises(ValueError, match="bias dtype"):
        fno.channel_mix(x, A, torch.zeros(4, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError, match="add shape"):
        fno.channel_mix(x, A, None, torch.zeros(2, 4, 6, device=DEV))
    prm = fno.NormParams("rms", 1e-5)
    with pytest.raises(ValueError, match="v shape"):
        fno.norm_residual(x, torch.zeros(2, 3, 6, device=DEV), prm)
    with pytest.raises(ValueError, match="gate shape"):
        fno.norm_residual(x, x.clone(), fno.NormParams("rms", 1e-5, gate=torch.zeros(3, device=DEV)))


def test_backward_twice_is_refused():
    x = torch.randn(1, 4, 32, device=DEV, requires_grad=True)
    A = torch.randn(4, 4, device=DEV)
    (g,) = torch.autograd.grad(fno.channel_mix(x, A, act=1).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


# ------------------------------------------------------------------ graphs

@pytest.mark.parametrize("dtype", DTYPES)
def test_training_step_from_a_captured_graph(dtype):
    """Mix, norms and their backward passes as one graph, replayed on new inputs with eager work between."""
    B, C, P = 3, 40, 1000
    rng = np.random.default_rng(31)
    make = lambda *s, scale=1.0: stored(rng, s, dtype, scale)[0].to(DEV)  # noqa: E731
    x, add, xr, gy, gu = (make(B, C, P) for _ in range(5))
    A, bias = make(C, C, scale=C ** -0.5), make(C)
    p = {k: make(B, C) if k == "gate" else make(C) for k in NORM_NAMES}

    def buffers():
        e = lambda *s: torch.zeros(s, dtype=DT[dtype], device=DEV)  # noqa: E731
        return dict(v=e(B, C, P), y=e(B, C, P), u=e(B, C, P), gx=e(B, C, P), gv=e(B, C, P), g=e(B, C, P), gA=e(C, C),
                    gb=e(C), ga=e(B, C, P), kept=fno.fno_channel_mix_saved_empty(x, C, 1, True),
                    ws=fno.fno_channel_mix_workspace_empty(x, C), nkept=fno.fno_norm_residual_saved_empty(x),
                    nws=fno.fno_norm_residual_workspace_empty(x), gp={k: torch.zeros_like(t) for k, t in p.items()})

    def step(b):
        prm, grads = fno.NormParams("layer", 1e-5, **p), fno.NormGrads(**b["gp"])
        fno.fno_channel_mix_save(x, A, bias, add, b["v"], b["kept"], 1)
        fno.fno_norm_residual_save(prm, xr, b["v"], b["y"], b["u"], b["nkept"])
        fno.fno_norm_residual_backward_saved(prm, b["nkept"], gy, gu, b["gx"], b["gv"], grads, b["nws"])
        fno.fno_channel_mix_backward_saved(b["kept"], A, bias, b["gv"], b["g"], b["gA"], b["gb"], b["ga"], b["ws"], 1,
                                           True)

    eager, held = buffers(), buffers()
    step(eager)  # kernels are loaded and attributes set before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for _ in range(3):
        for t in (x, add, xr, gy, gu):
            t.copy_(torch.randn(t.shape, device=DEV))
        graph.replay()
        step(eager)
        torch.cuda.synchronize()
        for k in ("v", "y", "u", "gx", "gv", "g", "gA", "gb", "ga"):
            assert torch.equal(held[k], eager[k]), k
        for k in p:
            assert torch.equal(held["gp"][k], eager["gp"][k]), k


# ----------------------------------------------------------------- example

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_conditioned_fno2d.py")
    spec = importlib.util.spec_from_file_location("train_conditioned_fno2d", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("keep", ["8bit", "whole"])
def test_example_trains(keep):
    losses = _example().train(steps=60, batch=8, grid=(32, 32), channels=16, modes=(8, 8), blocks=2, lr=4e-3, keep=keep)
    assert np.isfinite(losses).all()
    # an untrained network is off by about the norm of the field itself; halved is far
    # outside the spread of fresh batches
    assert np.mean(losses[-5:]) < 0.5 * np.mean(losses[:2])
