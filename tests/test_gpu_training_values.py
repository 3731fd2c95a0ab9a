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
