"""Group norm of values that differ little from a large level: a group that is read once has the mean that 64 bits give, rounded once."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import block as ref
from test_gpu_group_norm import EPS, run
from training_util import CHAIN, DT, f64, half_step, stored

pytestmark = pytest.mark.gpu
# (B, C, P, groups), held by teams of 8, 16, 64, 256 and 1024 threads, the last with eight chunks each: whole rows and
# ragged ones, tokens
HELD = [(3, 4, 12, 2), (4, 40, 1, 2), (2, 12, 100, 4), (9, 257, 1, 1), (2, 48, 33, 3), (5, 32, 100, 1), (100, 61, 97, 1),
        (100, 24, 2048, 3), (97, 8, 4090, 1)]
# groups that no team holds
SPLIT = [(1, 61, 97, 1), (2, 6, 40001, 2), (1, 512, 300, 1), (1, 4100, 20, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("level", [1000.1, -3.3, 1e-3])
@pytest.mark.parametrize("shape", HELD + SPLIT, ids=str)
def test_constant_groups(shape, level, last, dtype):
    """No deviation: y is the bias, rounded once, and x^ counts nothing in gw."""
    B, C, P, G = shape
    rng = np.random.default_rng(1)
    x = torch.full((B, P, C) if last else (B, C, P), level, dtype=DT[dtype])
    w, b, gy = stored(rng, (C,), dtype), stored(rng, (C,), dtype), stored(rng, tuple(x.shape), dtype)
    y, stats, gx, gw, gb = run(dtype, B, C, P, G, last, 0, None, dict(x=(x, None), gy=gy, w=w, b=b))
    assert (y == b[0].to(y.device).view(1, 1, C) if last else y == b[0].to(y.device).view(1, C, 1)).all()
    assert (stats[..., 0] == x.flatten()[0].float().item()).all() and (gw == 0).all()
    assert ((stats[..., 1].double() * EPS ** 0.5 - 1).abs() <= 4 * 2.0 ** -24).all()


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("level,spread", [(1000.1, 1e-2), (-3.3, 1e-4), (30.7, 1.0)])
@pytest.mark.parametrize("shape", HELD + SPLIT, ids=str)
def test_small_deviations(shape, level, spread, last):
    """y is off by what half a step of the mean comes to (a group in pieces: half a step each time that pieces are
    joined, 64 of them at most count, as in CHAIN), and by CHAIN of its own size."""
    B, C, P, G = shape
    rng = np.random.default_rng(2)
    x = torch.from_numpy(level + spread * rng.standard_normal((B, P, C) if last else (B, C, P))).float()
    w, b, gy = stored(rng, (C,), "f32"), stored(rng, (C,), "f32"), stored(rng, tuple(x.shape), "f32")
    y, stats, *_ = run("f32", B, C, P, G, last, 0, None, dict(x=(x, None), gy=gy, w=w, b=b))
    ry, mean, r, _ = ref.group_norm(x.double().numpy(), G, EPS, w[1], b[1], 0, last)
    per = lambda v: (v[None, None, :] if last else v[None, :, None])  # noqa: E731
    of = lambda s: per(np.ones(C)) * (np.repeat(s, C // G, 1)[:, None, :] if last else np.repeat(s, C // G, 1)[:, :, None])  # noqa: E731
    # half a step of the mean, and CHAIN of the deviations that corrected it: 16 standard ones at most
    m_off = (2.0 ** -24 if shape in HELD else CHAIN) * abs(mean) * 1.001 + CHAIN * 16 * spread
    assert (abs(f64(stats)[..., 0] - mean) <= m_off).all()
    # the terms of y: x^ w and b
    size = abs(ry - per(b[1])) + abs(per(b[1]))
    bound = of(m_off * r) * abs(per(w[1])) + CHAIN * size + half_step("f32") * abs(ry)
    assert (abs(f64(y) - ry) <= bound).all()


@pytest.mark.parametrize("last", [False, True])
@pytest.mark.parametrize("shape", HELD, ids=str)
def test_constant_groups_whose_squares_overflow(shape, last):
    """At 1e30 a step of the level squared is past fp32: y is the bias all the same."""
    B, C, P, G = shape
    rng = np.random.default_rng(3)
    x = torch.full((B, P, C) if last else (B, C, P), 1.1e30)
    w, b, gy = stored(rng, (C,), "f32"), stored(rng, (C,), "f32"), stored(rng, tuple(x.shape), "f32")
    y, *_ = run("f32", B, C, P, G, last, 0, None, dict(x=(x, None), gy=gy, w=w, b=b))
    assert (y == b[0].to(y.device).view((1, 1, C) if last else (1, C, 1))).all()
