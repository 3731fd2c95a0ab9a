"""GPU values of the training channel mix at the ends of its range: sums that pass the
largest fp32 number, GELU far out on the left, and gradients that cancel."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from training_util import DT

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]
DEV = "cuda:0"


def _run(x, A, bias, add, gy, act=1):
    """(y, gx, gA, gbias, gadd) of device tensors."""
    O = A.shape[0]
    y = torch.empty_like(gy)
    saved = fno.fno_channel_mix_saved_empty(x, O, act, add is not None)
    fno.fno_channel_mix_save(x, A, bias, add, y, saved, act)
    gx, gA, gbias, gadd = torch.empty_like(x), torch.empty_like(A), torch.empty_like(bias), torch.empty_like(gy)
    fno.fno_channel_mix_backward_saved(saved, A, bias, gy, gx, gA, gbias, gadd if add is not None else None,
                                       fno.fno_channel_mix_workspace_empty(x, O), act, add is not None)
    return y, gx, gA, gbias, gadd


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [3, 40])
def test_mix_slope_of_infinite_z(dtype, channels):
    """z = +-infinity from finite fields (an infinite bias; in fp32 and bf16 also a product past the
    largest number): GELU is infinite or 0 there, its derivative 1 or 0."""
    rng = np.random.default_rng(channels)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DT[dtype]).to(DEV)  # noqa: E731
    x, A, bias, add, gy = t(2, 5, 100), t(channels, 5), t(channels), t(2, channels, 100), t(2, channels, 100)
    bias[0], bias[1] = float("inf"), -float("inf")
    y, gx, gA, gbias, gadd = _run(x, A, bias, add, gy)
    assert (y[:, 0] == float("inf")).all() and (y[:, 1] == 0).all()
    assert torch.equal(gadd[:, 0], gy[:, 0]) and (gadd[:, 1] == 0).all()
    assert all(torch.isfinite(g).all() for g in (gx, gA, gbias))
    assert (gA[1] == 0).all() and gbias[1] == 0
    if dtype == "f16":
        return  # its products stay far below the largest fp32 number
    x, A, bias = x[:, :1].abs().contiguous() + 1, torch.full_like(A[:, :1], 3.0).contiguous(), torch.zeros_like(bias)
    big = x * 1e38
    A[1] = -3.0
    x = big.clamp(2e38, 3e38)
    y, gx, gA, gbias, gadd = _run(x, A, bias, add, gy)
    assert (y[:, 0] == float("inf")).all() and (y[:, 1] == 0).all()
    assert torch.equal(gadd[:, 0], gy[:, 0]) and (gadd[:, 1] == 0).all()
    assert torch.isfinite(gx).all() and torch.isfinite(gbias).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_mix_gelu_of_every_storage_value(dtype):
    """GELU of all storage values in [-8, 8] (z = add). The normal tail q is off by at most 1e-8 (its fit)
    and about ten roundings, and v^2 / 2 carries two more into the exponential: |v| times that, and the
    rounding of the result, bound the error, so a small GELU far out on the left keeps its digits."""
    z = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    z = z[torch.isfinite(z) & (z.abs() <= 8)]
    n = z.numel()
    z64 = z.double()
    ref = z64 * torch.special.ndtr(z64)
    add = z.view(1, 1, n).to(DEV)
    one = torch.zeros(1, 1, n, dtype=DT[dtype], device=DEV)
    y, *_ = _run(one, torch.zeros(1, 1, dtype=DT[dtype], device=DEV), torch.zeros(1, dtype=DT[dtype], device=DEV), add,
                 add.clone())
    q = torch.special.ndtr(-z64.abs())
    step = torch.finfo(DT[dtype]).eps / 2 * ref.abs() + (2.0 ** -25 if dtype == "f16" else 2.0 ** -134)
    bound = step * (1 + 2.0 ** -10) + z64.abs() * (1e-8 + (10 + z64 ** 2) * 2.0 ** -24 * q) + 2.0 ** -24 * ref.abs()
    off = (y.view(-1).cpu().double() - ref).abs()
    assert (off <= bound).all(), f"over by {float((off / bound).max()):.3g} at {float(z64[(off / bound).argmax()])}"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("channels", [2, 16, 24, 64, 100])
def test_mix_gradients_that_cancel(dtype, channels):
    """Pairs of output channels with opposite weights and nearly equal z: gx and gA are small differences of
    gz, an fp32 value whatever the fields' type. Bounds: z is off by 2 2^-24 max(|z|, 1) and the derivative, of slope
    at most 0.8, by 12 2^-24 more; a sum of c_out (or of all pixels') products adds a rounding of its
    partial sums, at most the sizes' sum, for each of its steps in a row, fewer than 8; sizes at most |gy| 1.13."""
    rng = np.random.default_rng(channels)
    P, half = 192, channels // 2
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DT[dtype])  # noqa: E731
    # add in steps of 2^-5, which 8 bits keep as every block's largest is 2; the partner's is a step off
    add1 = (t(1, half, P).double() * 0.5).to(DT[dtype])
    add1 = (torch.round(add1.double() * 32) / 32).to(DT[dtype])
    add1[..., ::32] = 2.0
    add1 = add1.clamp(-2, 2)
    add2 = (add1.double() + 2.0 ** -5).clamp(-2, 2).to(DT[dtype])
    add = torch.cat([add1, add2], 1)
    A = torch.cat([torch.ones(half, 1), -torch.ones(half, 1)]).to(DT[dtype])
    bias = torch.cat([torch.zeros(half), 2 * torch.ones(half)]).to(DT[dtype])  # with x = 1, z = 1 + add for both
    gy = t(1, half, P)
    gy = torch.cat([gy, gy], 1)
    x = torch.ones(1, 1, P, dtype=DT[dtype])
    _, gx, gA, gbias, gadd = _run(*(s.to(DEV) for s in (x, A, bias, add, gy)))
    z = add.double() + 1
    slope = torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    gz = gy.double() * slope
    want = (A.double()[None] * gz).sum(1, keepdim=True)
    size = gy.double().abs()
    assert float(want.abs().mean() / size.sum(1).mean()) < 0.05  # they do cancel
    tol = ((0.8 * 2 * 3 + 12) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * 1.13 * size).sum(1, keepdim=True)
    half_step = torch.finfo(DT[dtype]).eps / 2
    off = (gx.cpu().double() - want).abs() - half_step * (1 + 2.0 ** -10) * want.abs() - tol
    assert (off <= 0).all(), f"gx over by {float(off.max()):.3g}, tolerance {float(tol.max()):.3g}"
    sums = gz.sum(2)[0]
    tol = ((0.8 * 2 * 3 + 12) * 2.0 ** -24 * size + 8 * 2.0 ** -24 * 1.13 * size).sum(2)[0]
    off = (gA.cpu().double()[:, 0] - sums).abs() - half_step * (1 + 2.0 ** -10) * sums.abs() - tol
    assert (off <= 0).all(), f"gA over by {float(off.max()):.3g}, tolerance {float(tol.max()):.3g}"
