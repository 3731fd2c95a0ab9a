"""GPU parity of group norm with activation and dropout, forward and backward, with the
float64 definition (oracle/block.py), at the sizes where its kernels change and values where it
can go wrong."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import block as ref
from training_util import CHAIN, DT, close, f64, half_step, stored

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
# (B, C, P, groups): groups of one value, teams of 16, 64, 256 and 1024 threads, chunk and
# row ends, groups past a workgroup's registers with short, middle and long rows, with
# more channels than 256 chunks, many samples, tokens, teams of 1024 for enough groups, many channels of long rows
SHAPES = [(1, 1, 1, 1), (2, 4, 256, 2), (1, 1, 2, 1), (5, 64, 1, 8), (3, 6, 2, 3), (2, 48, 33, 3), (1, 61, 97, 1),
          (2, 12, 100, 4), (9, 257, 1, 1), (1, 96, 1000, 3), (2, 48, 3721, 3), (1, 3, 70001, 1), (2, 512, 300, 1),
          (1, 4096, 20, 2), (300, 40, 1, 5), (1, 8192, 1, 1), (2, 8192, 9, 4), (70, 24, 50, 24), (3, 2, 40000, 2),
          (2, 1000, 3, 1), (17, 16, 16, 2), (1, 6, 32771, 2), (24, 32, 1500, 4), (12, 64, 4500, 8),
          (12, 64, 2101, 8), (1, 1030, 2060, 1)]


def case(dtype, B, C, P, last, seed, mean=0.5):
    rng = np.random.default_rng(seed)
    shape = (B, P, C) if last else (B, C, P)
    x, x64 = stored(rng, shape, dtype)
    if mean:
        level = rng.standard_normal((B, 1, C) if last else (B, C, 1)) * mean
        x = (x.double() + torch.from_numpy(level)).to(DT[dtype])
        x64 = x.double().numpy()
    gy, gy64 = stored(rng, shape, dtype, 0.5)
    w, w64 = stored(rng, (C,), dtype, 0.3)
    b, b64 = stored(rng, (C,), dtype, 0.3)
    w, w64 = (w.double() + 1).to(DT[dtype]), (w.double() + 1).to(DT[dtype]).double().numpy()
    return dict(x=(x, x64), gy=(gy, gy64), w=(w, w64), b=(b, b64))


def run(dtype, B, C, P, G, last, act, drop, c, absent=False, eps=EPS):
    flat = (B, C) if P == 1 else c["x"][0].shape
    x, gy = c["x"][0].to(DEV).view(flat), c["gy"][0].to(DEV).view(flat)
    w, b = (None, None) if absent else (c["w"][0].to(DEV), c["b"][0].to(DEV))
    prm = fno.GroupNormParams(G, eps, w, b, act=act, channels_last=last)
    ws = torch.full_like(fno.fno_group_norm_workspace_empty(x, G, last), 255)
    y, gx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    gw, gb = (None, None) if absent else (torch.full_like(w, 7.0), torch.full_like(b, 7.0))
    stats = torch.full_like(fno.fno_group_norm_stats_empty(x, G), 7.0)
    fno.fno_group_norm(prm, x, y, stats, ws, drop)
    ws.fill_(255)
    fno.fno_group_norm_backward(prm, x, stats, gy, gx, gw, gb, ws, drop)
    shape = c["x"][0].shape
    return y.view(shape), stats, gx.view(shape), gw, gb


def compare(dtype, B, C, P, G, last, act, drop, c, got, absent=False, eps=EPS):
    y, stats, gx, gw, gb = got
    f = 1.0 if drop is None else ref.drop_factor(B, C, P, last, drop.p, drop.seed, drop.offset, drop.unit)
    w, b = (None, None) if absent else (c["w"][1], c["b"][1])
    x, gy = c["x"][1], c["gy"][1]
    ry, mean, r, size = ref.group_norm(x, G, eps, w, b, act, last, f)
    close("y", y, ry, dtype, size=size)
    st = f64(stats)
    level = np.sqrt((ref._grouped(x, G, last)[0] ** 2).mean(ref._grouped(x, G, last)[1]))
    assert (abs(st[..., 0] - mean) <= CHAIN * level).all()
    # the variance is off by CHAIN of itself and by what an error of the mean of 2^-23 of the level adds
    assert (abs(st[..., 1] / r - 1) <= CHAIN + (2.0 ** -23 * level * r) ** 2).all()
    (rx, rw, rb), (sx, sw, sb) = ref.group_norm_backward(x, G, eps, w, b, act, last, gy, f)
    close("gx", gx, rx, dtype, size=sx)
    if not absent:
        close("gw", gw, rw, dtype, size=sw)
        close("gb", gb, rb, dtype, size=sb)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_group_norm(dtype, last, shape):
    B, C, P, G = shape
    i = SHAPES.index(shape)
    for act, drop in ((i % 3, None), ((i + 1) % 3, fno.Dropout(0.3, 77 + i, i << 33, unit=["element", "channel", "sample"][i % 3]))):
        c = case(dtype, B, C, P, last, i)
        compare(dtype, B, C, P, G, last, act, drop, c, run(dtype, B, C, P, G, last, act, drop, c))


@pytest.mark.parametrize("unit", ["element", "channel", "sample"])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(3, 10, 21, 5), (3, 30, 4099, 3), (4, 40, 1, 2)], ids=str)
def test_every_activation_and_unit(shape, last, act, unit):
    B, C, P, G = shape
    for dtype in ("f32", "f16"):
        c = case(dtype, B, C, P, last, act)
        d = fno.Dropout(0.5, 3, 4, unit=unit)
        compare(dtype, B, C, P, G, last, act, d, c, run(dtype, B, C, P, G, last, act, d, c))


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 6, 40, 3), (2, 6, 70000, 2), (3, 33, 1, 3)], ids=str)
def test_absent_parameters(shape, last):
    B, C, P, G = shape
    c = case("bf16", B, C, P, last, 1)
    compare("bf16", B, C, P, G, last, 2, None, c, run("bf16", B, C, P, G, last, 2, None, c, absent=True), absent=True)


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 8, 50, 2), (2, 8, 20000, 2), (2, 64, 1, 4)], ids=str)
def test_wanted_gradients_alone(shape, last):
    """Each gradient by itself is that of all together, bit for bit."""
    B, C, P, G = shape
    c = case("f32", B, C, P, last, 2)
    flat = (B, C) if P == 1 else c["x"][0].shape
    x, gy, w, b = (c[k][0].to(DEV) for k in ("x", "gy", "w", "b"))
    x, gy = x.view(flat), gy.view(flat)
    prm = fno.GroupNormParams(G, EPS, w, b, act=1, channels_last=last)
    stats, ws = fno.fno_group_norm_stats_empty(x, G), fno.fno_group_norm_workspace_empty(x, G, last)
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    fno.fno_group_norm(prm, x, y, stats, ws)
    fno.fno_group_norm(prm, x, y2, None, ws)  # without statistics
    assert torch.equal(y, y2)
    want = [torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)]
    fno.fno_group_norm_backward(prm, x, stats, gy, *want, ws)
    for i in range(3):
        one = [None, None, None]
        one[i] = torch.full_like(want[i], 9.0)
        fno.fno_group_norm_backward(prm, x, stats, gy, *one, ws)
        assert torch.equal(one[i], want[i])
    again = [torch.empty_like(t) for t in want]
    fno.fno_group_norm_backward(prm, x, stats, gy, *again, ws)
    assert all(torch.equal(a, b) for a, b in zip(want, again))


BIG = [(2, 8, 50, 2), (1, 4, 60001, 2), (2, 64, 1, 4), (1, 32, 5000, 2)]


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", BIG, ids=str)
@pytest.mark.parametrize("mean", [1000.0, -30.0])
def test_levels_far_from_zero(shape, last, mean):
    """A level of a thousand deviations costs the digits that fp32 loses in x - mean, no more."""
    B, C, P, G = shape
    c = case("f32", B, C, P, last, 4, mean=0)
    x = (c["x"][0].double() + mean).float()
    c["x"] = (x, x.double().numpy())
    compare("f32", B, C, P, G, last, 0, None, c, run("f32", B, C, P, G, last, 0, None, c))


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", BIG, ids=str)
def test_outliers(shape, last):
    """One value of a group a million times the others, at the places where sums start or end."""
    B, C, P, G = shape
    for at in (0, 1, max(P, C // G) - 1 if P == 1 else P - 1):
        c = case("f32", B, C, P, last, 5, mean=0)
        x = c["x"][0].clone()
        if P == 1:
            x.view(B, C)[0, at] = 1e6
        else:
            x[(0, at, 0) if last else (0, 0, at)] = 1e6
        c["x"] = (x, x.double().numpy())
        compare("f32", B, C, P, G, last, 0, None, c, run("f32", B, C, P, G, last, 0, None, c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", BIG, ids=str)
def test_constant_groups(shape, last, dtype):
    """No deviation: y is act(bias), whatever the level."""
    B, C, P, G = shape
    c = case(dtype, B, C, P, last, 6)
    x = torch.full(c["x"][0].shape, 3.140625, dtype=DT[dtype])
    c["x"] = (x, x.double().numpy())
    y, stats, gx, gw, gb = run(dtype, B, C, P, G, last, 0, None, c)
    # the mean is a sum of equal values over their number: off by CHAIN of it at most, times r = eps^-1/2
    b = c["b"][1][None, None, :] if last else c["b"][1][None, :, None]
    w = abs(c["w"][1][None, None, :] if last else c["w"][1][None, :, None])
    bound = half_step(dtype) * abs(b) * 1.001 + CHAIN * 3.15 * EPS ** -0.5 * w + CHAIN
    assert (abs(f64(y) - b) <= bound).all()
    assert np.isfinite(f64(gx)).all() and np.isfinite(f64(gw)).all()


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(3, 8, 50, 2), (3, 4, 40001, 2), (3, 64, 1, 4), (3, 16, 9, 2)], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_poison_stays_in_its_group(shape, last, bad):
    B, C, P, G = shape
    c = case("f32", B, C, P, last, 7)
    x = c["x"][0].clone()
    x[(1, P // 2, C - 1) if last else (1, C - 1, P // 2)] = bad
    c2 = dict(c, x=(x, None))
    y0, s0, gx0, _, _ = run("f32", B, C, P, G, last, 1, None, c)
    y, s, gx, gw, gb = run("f32", B, C, P, G, last, 1, None, c2)
    hit = torch.zeros(x.shape, dtype=torch.bool)
    lo = C - C // G
    if last:
        hit[1, :, lo:] = True
    else:
        hit[1, lo:] = True
    hit = hit.to(DEV)
    assert torch.isnan(y[hit]).all() and torch.isnan(gx[hit]).all()
    assert torch.equal(y[~hit], y0[~hit]) and torch.equal(gx[~hit], gx0[~hit])
    assert torch.isfinite(gw[:lo]).all() and torch.isnan(gw[lo:]).all()


@pytest.mark.parametrize("last", [False, True])
def test_dropped_gradients_do_not_poison(last):
    """A dropped value's gradient does not count, whatever it is."""
    B, C, P, G = 2, 8, 300, 2
    c = case("f32", B, C, P, last, 8)
    d = fno.Dropout(0.5, 5)
    f = ref.drop_factor(B, C, P, last, d.p, d.seed)
    gy = c["gy"][0].clone()
    gy[torch.from_numpy(f == 0)] = float("nan")
    c2 = dict(c, gy=(gy, c["gy"][1]))
    compare("f32", B, C, P, G, last, 1, d, c, run("f32", B, C, P, G, last, 1, d, c2))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 12, 33, 3), (2, 3, 21, 1), (1, 9, 20001, 3), (3, 20, 1, 4)], ids=str)
def test_guards(dtype, last, shape):
    """Nothing is written beside the outputs, the workspace's end included."""
    B, C, P, G = shape
    c = case(dtype, B, C, P, last, 9)
    n = B * C * P
    x, gy, w, b = (c[k][0].to(DEV) for k in ("x", "gy", "w", "b"))
    room = lambda k, dt: torch.full((k + 128,), 3.0, dtype=dt, device=DEV)  # noqa: E731
    bufs = {k: room(m, DT[dtype]) for k, m in (("y", n), ("gx", n), ("gw", C), ("gb", C))}
    bufs["stats"] = room(B * G * 2, torch.float32)
    part = {k: v[64:-64] for k, v in bufs.items()}
    size = fno.fno_group_norm_workspace_bytes(B, C, P, G, last, dtype)
    wbuf = torch.full((size + 512,), 99, dtype=torch.uint8, device=DEV)
    ws = wbuf[256:256 + size]
    prm = fno.GroupNormParams(G, EPS, w, b, act=1, channels_last=last)
    y, gx = part["y"].view(x.shape), part["gx"].view(x.shape)
    stats = part["stats"].view(B, G, 2)
    fno.fno_group_norm(prm, x, y, stats, ws)
    fno.fno_group_norm_backward(prm, x, stats, gy, gx, part["gw"], part["gb"], ws)
    for k, v in bufs.items():
        assert (v[:64] == 3).all() and (v[-64:] == 3).all(), k
    assert (wbuf[:256] == 99).all() and (wbuf[256 + size:] == 99).all()


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", [(2, 12, 33, 3), (2, 6, 40000, 2)], ids=str)
def test_graph_and_stream(last, shape):
    B, C, P, G = shape
    c = case("f16", B, C, P, last, 10)
    x, gy, w, b = (c[k][0].to(DEV) for k in ("x", "gy", "w", "b"))
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    prm = fno.GroupNormParams(G, EPS, w, b, act=2, channels_last=last)
    out = [torch.empty_like(t) for t in (x, x, w, b)]
    stats, ws = fno.fno_group_norm_stats_empty(x, G), fno.fno_group_norm_workspace_empty(x, G, last)

    def step_of(d, o):
        fno.fno_group_norm(prm, x, o[0], stats, ws, d)
        fno.fno_group_norm_backward(prm, x, stats, gy, o[1], o[2], o[3], ws, d)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step_of(fno.Dropout(0.2, 1, 50, step=step), out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step_of(fno.Dropout(0.2, 1, 50, step=step), out)
    for i in range(3):
        step.fill_(i)
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = [torch.empty_like(t) for t in out]
        step_of(fno.Dropout(0.2, 1, 50 + i), want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def _torch_form(x, w, b, G, act, last, f, eps=EPS):
    B, C = x.shape[0], x.shape[-1 if last else 1]
    h = x.reshape(B, -1, G, C // G) if last else x.reshape(B, G, C // G, -1)
    over = (1, 3) if last else (2, 3)
    h = h - h.mean(over, keepdim=True)
    h = (h / torch.sqrt((h * h).mean(over, keepdim=True) + eps)).reshape(x.shape)
    at = (lambda p: p) if last else (lambda p: p.view(1, C, *([1] * (x.dim() - 2))))
    z = h * at(w) + at(b)
    z = [z, z * torch.special.ndtr(z), z * torch.sigmoid(z)][act]
    return z * f


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("grid", [(5, 7), (3, 4, 5), ()], ids=str)
def test_autograd(last, grid):
    B, C, G = 2, 12, 3
    rng = np.random.default_rng(1)
    P = int(np.prod(grid)) if grid else 1
    shape = (B, *grid, C) if last else (B, C, *grid)
    t = lambda s: torch.from_numpy(rng.standard_normal(s)).float().to(DEV).requires_grad_()  # noqa: E731
    x, w, b = t(shape), t((C,)), t((C,))
    d = fno.Dropout(0.3, 8, unit="element")
    f = torch.from_numpy(np.array(ref.drop_factor(B, C, P, last, d.p, d.seed)).reshape(shape)).to(DEV)
    y = fno.group_norm(x, fno.GroupNormParams(G, EPS, w, b, act=1, channels_last=last), d)
    gy = torch.randn_like(y)
    y.backward(gy)
    leaves = [v.detach().double().requires_grad_() for v in (x, w, b)]
    yr = _torch_form(*leaves, G, 1, last, f)
    yr.backward(gy.double())
    assert (y.double() - yr).abs().max() < 1e-5
    for a, r in zip((x, w, b), leaves):
        assert (a.grad.double() - r.grad).abs().max() <= 1e-5 * (1 + r.grad.abs().max())


def test_autograd_of_strided_inputs_and_frozen_parameters():
    C, G = 12, 3
    base = torch.randn(2, 35, C, device=DEV, requires_grad=True)
    w, b = torch.randn(C, device=DEV), torch.randn(2 * C, device=DEV, requires_grad=True)
    x = base.transpose(1, 2)  # strided
    y = fno.group_norm(x, fno.GroupNormParams(G, EPS, w, b[::2], act=2))
    y.sum().backward()  # a broadcast gradient
    xr, br = base.detach().double().requires_grad_(), b.detach().double().requires_grad_()
    _torch_form(xr.transpose(1, 2), w.double(), br[::2], G, 2, False, 1.0).sum().backward()
    assert (base.grad.double() - xr.grad).abs().max() < 1e-4 and (b.grad.double() - br.grad).abs().max() < 1e-4
    with torch.no_grad():
        y2 = fno.group_norm(x, fno.GroupNormParams(G, EPS, w, b[::2], act=2))
    assert torch.equal(y, y2)


def test_captured_backward_of_leaves_that_an_eager_graph_holds():
    """Refused, not the end of the process; once the eager graph is gone the step can be captured."""
    x = torch.randn(2, 8, 40, device=DEV, requires_grad=True)
    w = torch.ones(8, device=DEV, requires_grad=True)
    b = torch.zeros(8, device=DEV, requires_grad=True)
    prm = fno.GroupNormParams(2, EPS, w, b, act=1)
    d = fno.Dropout(0.5, 1)
    eager = fno.dropout_residual(fno.group_norm(x, prm, d), d, x)
    gy = torch.randn_like(eager)
    for call in (lambda: fno.group_norm(x, prm, d), lambda: fno.dropout_residual(x, d)):
        with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
    want = torch.autograd.grad(eager, (x, w, b), gy)
    del eager
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = torch.autograd.grad(fno.dropout_residual(fno.group_norm(x, prm, d), d, x), (x, w, b), gy)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, r) for a, r in zip(got, want))
