"""What the differentiable training operators do where no gradient is wanted."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from spectral_convolution_amd import _training as ops
from training_util import DT, norm_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P", [None, 200])
@pytest.mark.parametrize("how", ["no_grad", "no_leaf"])
def test_norm_keeps_nothing_without_a_gradient(dtype, P, how, monkeypatch):
    c, prm = norm_case(dtype, 3, 24, P, seed=21)
    x, v = (c[k][0].to("cuda") for k in ("x", "v"))
    p = {k: t[0].to("cuda") for k, t in prm.items()}
    y, u = fno.norm_residual(x.clone().requires_grad_(), v, fno.NormParams("layer", 1e-5, **p))

    def refuse(*_):
        raise AssertionError("a checkpoint was made")

    monkeypatch.setattr(ops, "fno_norm_residual_saved_empty", refuse)
    monkeypatch.setattr(ops, "fno_norm_residual_save", refuse)
    if how == "no_grad":
        with torch.no_grad():
            got = fno.norm_residual(x.clone().requires_grad_(), v, fno.NormParams("layer", 1e-5, **p))
    else:
        got = fno.norm_residual(x, v, fno.NormParams("layer", 1e-5, **p))
    assert torch.equal(got[0], y) and torch.equal(got[1], u) and not got[0].requires_grad
    with pytest.raises(AssertionError, match="checkpoint"):
        fno.norm_residual(x, v, fno.NormParams("layer", 1e-5, **{**p, "gate": p["gate"].requires_grad_()}))


@pytest.mark.parametrize("dtype", list(DT))
def test_mix_is_the_same_without_a_gradient(dtype):
    rng = np.random.default_rng(22)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(DT[dtype]).to("cuda")  # noqa: E731
    x, A, b, add = t(2, 20, 11, 13), t(24, 20), t(24), t(2, 24, 11, 13)
    y = fno.channel_mix(x, A.requires_grad_(), b, add, act=1)
    with torch.no_grad():
        z = fno.channel_mix(x, A, b, add, act=1)
    assert y.requires_grad and not z.requires_grad and torch.equal(y, z)
