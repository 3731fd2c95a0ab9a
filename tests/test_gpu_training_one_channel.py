"""The layer norm over a single channel, on tokens and fields."""

import pytest
import torch

import training_ref64 as r64
from test_gpu_training import _run
from training_util import DT, NORM_NAMES

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P", [None, 90])
def test_layer_norm_of_one_channel(dtype, P):
    """One channel has no deviation from its mean: v^ = y^ = 0, so y = x + scale gate b_post, u = b_pre, nothing
    flows back through a norm, and all of it exactly (y: one rounding of the product and one of the result)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    shape = (7, 1) if P is None else (7, 1, P)

    def stored(s, scale, mean=0.0):
        t = (torch.randn(s, generator=gen, device="cuda") * scale + mean).to(DT[dtype])
        return t, t.double()

    c = {k: stored(shape, 2.0) for k in ("x", "v", "gy", "gu")}
    prm = {k: stored((7, 1) if k == "gate" else (1,), 0.3, 1.0) for k in NORM_NAMES}
    for saved_form in (False, True):
        y, u, gx, gv, grads = _run(dtype, "layer", c, prm, saved_form)
        sg = prm["scale"][1] * prm["gate"][1] * prm["b_post"][1]
        want = c["x"][1] + (sg if P is None else sg[..., None])
        r64.close("y", y, want, dtype)
        assert torch.equal(u, prm["b_pre"][0].expand(shape) if P is None else prm["b_pre"][0][:, None].expand(shape))
        assert torch.equal(gx, c["gy"][0]) and (gv == 0).all()
        assert float(grads["w_post"].abs()) == 0 and float(grads["w_pre"].abs()) == 0
        n, s = prm["b_post"][1], (0,) if P is None else (0, 2)
        r64.close("g_b_pre", grads["b_pre"], c["gu"][1].sum(s), dtype, size=c["gu"][1].abs().sum(s))
        g = c["gy"][1] if P is None else c["gy"][1].sum(2)
        size = c["gy"][1].abs() if P is None else c["gy"][1].abs().sum(2)
        r64.close("g_gate", grads["gate"], g * prm["scale"][1] * n, dtype, size=size * (prm["scale"][1] * n).abs())
