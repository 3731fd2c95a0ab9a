"""GPU parity of dropout (alone, into a residual stream, in a captured graph and as an autograd
Function) with its definition (oracle/block.py): the mask has to be equal, values are one rounding."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import block as ref
from training_util import DT, f64, half_step, stored

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SEED, OFFSET = 0x9E3779B97F4A7C15, 0xFFFFFFFF7  # keys and counters past 32 bits
# (B, C, P): one value, chunk ends, whole workgroups and more, rows of one value, odd rows
SHAPES = [(1, 1, 1), (1, 3, 5), (2, 4, 256), (3, 7, 33), (5, 1001, 1), (1, 1, 8191), (4, 3, 3721), (7, 130, 9),
          (2, 64, 4096), (300, 40, 1), (33, 16, 2), (2, 520, 64)]


def field(rng, B, C, P, last, dtype, scale=1.0):
    shape = (B, C) if P == 1 else (B, P, C) if last else (B, C, P)
    t, v = stored(rng, shape, dtype, scale)
    return t.to(DEV), v


def factor(B, C, P, last, drop, shape):
    f = ref.drop_factor(B, C, P, last, drop.p, drop.seed, drop.offset, drop.unit)
    return np.array(np.broadcast_to(f, (B, P, C) if last else (B, C, P))).reshape(shape)


def check(got, x, v, f, dtype):
    """x + v f, rounded once: fp32 arithmetic in front adds its own two roundings."""
    y = v * f + (0 if x is None else x)
    bound = half_step(dtype) * abs(y) * (1 + 2.0 ** -10) + 2.0 ** -23 * (abs(v * f) + abs(y)) + (2.0 ** -25 if dtype == "f16" else 0)
    got = f64(got)
    assert np.isfinite(got).all() and (abs(got - y) <= bound).all()
    if x is None:
        assert (got[f == 0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("unit", ["element", "channel", "sample"])
@pytest.mark.parametrize("last", [False, True])
def test_dropout(dtype, unit, last):
    for i, (B, C, P) in enumerate(SHAPES):
        rng = np.random.default_rng(i)
        d = fno.Dropout([0.1, 0.5, 0.9][i % 3], SEED + i, OFFSET * (i + 1), unit=unit)
        v, v64 = field(rng, B, C, P, last, dtype)
        x, x64 = field(rng, B, C, P, last, dtype)
        f = factor(B, C, P, last, d, v64.shape)
        y = torch.full_like(v, 7.0)
        fno.fno_dropout_residual(d, None, v, y, channels_last=last)
        check(y, None, v64, f, dtype)
        y.fill_(7.0)
        fno.fno_dropout_residual(d, x, v, y, channels_last=last)
        check(y, x64, v64, f, dtype)


@pytest.mark.parametrize("p", [0.0, 1e-6, 1.0, 0.99999])
@pytest.mark.parametrize("unit", ["element", "channel", "sample"])
def test_ends_of_p(p, unit):
    rng = np.random.default_rng(3)
    v, v64 = field(rng, 3, 8, 700, False, "f32")
    x, x64 = field(rng, 3, 8, 700, False, "f32")
    d = fno.Dropout(p, 1, unit=unit)
    y = torch.empty_like(v)
    fno.fno_dropout_residual(d, x, v, y)
    check(y, x64, v64, factor(3, 8, 700, False, d, v64.shape), "f32")
    if p == 1.0:
        assert torch.equal(y, x)
    if p in (0.0, 1e-6):
        assert torch.equal(y, x + v)


@pytest.mark.parametrize("unit", ["element", "channel"])
def test_dropped_values_are_zero_whatever_they_were(unit):
    v = torch.full((4, 64, 100), float("nan"), device=DEV)
    v[1] = float("inf")
    d = fno.Dropout(0.5, 11, unit=unit)
    y = torch.empty_like(v)
    fno.fno_dropout_residual(d, None, v, y)
    f = factor(4, 64, 100, False, d, tuple(v.shape))
    got = y.cpu().numpy()
    assert (got[f == 0] == 0).all() and np.isnan(got[0][f[0] > 0]).all() and np.isinf(got[1][f[1] > 0]).all()


def test_one_drawing_does_not_depend_on_the_others():
    """Offsets and seeds give masks that agree no more often than by chance."""
    n = 1 << 20
    v = torch.ones(1, 1, n, device=DEV)
    masks = []
    for seed, offset in ((1, 0), (1, 1), (2, 0), (1, 1 << 32), (1 + (1 << 32), 0)):
        y = torch.empty_like(v)
        fno.fno_dropout_residual(fno.Dropout(0.5, seed, offset), None, v, y)
        masks.append((y != 0).flatten().float())
    for i, a in enumerate(masks):
        assert abs(a.mean().item() - 0.5) < 5 * 0.5 / n ** 0.5
        for b in masks[:i]:
            assert abs((a == b).float().mean().item() - 0.5) < 5 * 0.5 / n ** 0.5


def test_large_offsets_of_values():
    """Values past 2^32: the counter's high word and 64-bit addresses."""
    C, P = 33, 1 << 27
    v = torch.ones((1, C, P), dtype=torch.float16, device=DEV)
    y = torch.empty_like(v)
    fno.fno_dropout_residual(fno.Dropout(0.5, 5), None, v, y)
    n = 1 << 16
    w = ref.philox(np.arange(((C * P) - n) // 8, C * P // 8, dtype=np.uint64), 0, 5)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)
    assert ((y.view(-1)[-n:].cpu().numpy() != 0) == (bits >= 32768)).all()


def test_stream_step_and_graph():
    v = torch.randn(3, 50, 77, device=DEV)
    x = torch.randn_like(v)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    d = fno.Dropout(0.3, 9, 100, step=step)
    side = torch.cuda.Stream()
    y = torch.empty_like(v)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        fno.fno_dropout_residual(d, x, v, y)  # warm, and on another stream than the default one
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fno.fno_dropout_residual(d, x, v, y)
    seen = []
    for i in range(4):
        step.fill_(i)
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(y)
        fno.fno_dropout_residual(fno.Dropout(0.3, 9, 100 + i), x, v, want)
        assert torch.equal(y, want)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("residual", [False, True])
def test_autograd(residual):
    v = torch.randn(2, 6, 35, device=DEV, requires_grad=True)
    x = torch.randn(2, 6, 35, device=DEV, requires_grad=True) if residual else None
    d = fno.Dropout(0.4, 21)
    y = fno.dropout_residual(v, d, x)
    gy = torch.randn_like(y)
    y.backward(gy)
    f = torch.from_numpy(factor(2, 6, 35, False, d, tuple(v.shape))).float().to(DEV)
    assert torch.allclose(v.grad, gy * f, rtol=2.0 ** -22, atol=0)
    if residual:
        assert torch.equal(x.grad, gy)


def test_autograd_of_strided_and_broadcast_inputs():
    base = torch.randn(2, 35, 6, device=DEV, requires_grad=True)
    d = fno.Dropout(0.4, 21, unit="channel")
    y = fno.dropout_residual(base.transpose(1, 2), d)
    y.sum().backward()  # a broadcast gradient
    f = torch.from_numpy(factor(2, 6, 35, False, d, (2, 6, 35))).float().to(DEV)
    assert torch.allclose(base.grad, f.transpose(1, 2), rtol=2.0 ** -22, atol=0)


def test_guards():
    """Nothing is written beside y."""
    for B, C, P in SHAPES:
        n = B * C * P
        for dtype in ("f32", "bf16"):
            buf = torch.full((n + 64,), 3.0, dtype=DT[dtype], device=DEV)
            y = buf[16:16 + n].view(B, C, P)
            if y.data_ptr() % 16:
                pytest.fail("guard offset")
            v = torch.ones((B, C, P), dtype=DT[dtype], device=DEV)
            for unit in ("element", "channel", "sample"):
                fno.fno_dropout_residual(fno.Dropout(0.5, 1, unit=unit), None, v, y)
            assert (buf[:16] == 3).all() and (buf[16 + n:] == 3).all()
