"""Seeded cases of the training operators in float64 and in storage types, and
the error bounds their tests share."""

import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOW = {"f32": -126, "f16": -24, "bf16": -126}
NORM_NAMES = ("w_post", "b_post", "gate", "scale", "w_pre", "b_pre")

# Bounds. A result's last rounding is off by eps / 2 of the value. Before it, everything
# is fp32: an elementwise result passes through fewer than 64 roundings of 2^-24 of
# the largest quantity on its way, and a sum's partial sums (at most a few hundred
# terms deep in any one accumulator, error growing like the square root for the
# random signs used here, so fewer than 64 of them count) add 64 2^-24 of the sum
# of the terms' sizes.
CHAIN = 64 * 2.0 ** -24


def half_step(dtype):
    return float(torch.finfo(DT[dtype]).eps) / 2


def stored(rng, shape, dtype, scale=1.0, spread=False):
    """(tensor on the CPU in `dtype`, its values in float64)."""
    a = rng.standard_normal(shape) * scale
    if spread:  # rows of different strength, as channels have
        a = a * np.exp(0.5 * rng.standard_normal(shape[:-1] + (1,)))
    t = torch.from_numpy(a).to(DT[dtype])
    return t, t.double().numpy()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(name, got, ref, dtype, size=None, extra=0.0):
    """|got - ref| <= eps/2 |ref| + (CHAIN + extra) size, elementwise; size defaults to
    the larger of |ref| and its root mean square. fp16's subnormal step counts too."""
    got, ref = f64(got), np.asarray(ref)
    assert got.shape == ref.shape, name
    if size is None:
        size = np.maximum(abs(ref), np.sqrt(np.mean(ref ** 2)))
    step = 2.0 ** -25 if dtype == "f16" else 0.0
    bound = half_step(dtype) * abs(ref) * (1 + 2.0 ** -10) + (CHAIN + extra) * size + step
    off = abs(got - ref) - bound
    assert np.isfinite(got).all(), f"{name}: not finite"
    assert (off <= 0).all(), (f"{name}: off by {abs(got - ref).max():.3g}, {np.count_nonzero(off > 0)} of {off.size} "
                              f"over the bound by up to {off.max():.3g}")


def norm_case(dtype, B, C, P, seed=0, absent=(), mean=0.0):
    """Fields ([B][C][P], or [B][C] where P is None) and parameters."""
    rng = np.random.default_rng(seed)
    shape = (B, C) if P is None else (B, C, P)
    c = {"x": stored(rng, shape, dtype), "v": stored(rng, shape, dtype, 3.0),
         "gy": stored(rng, shape, dtype, 0.5), "gu": stored(rng, shape, dtype, 0.5)}
    if mean:
        t = (c["v"][0].double() + mean).to(DT[dtype])
        c["v"] = (t, t.double().numpy())
    prm = {}
    for k, (mid, dev, s) in {"w_post": (1.0, 0.2, (C,)), "b_post": (0.0, 0.1, (C,)), "gate": (0.5, 0.3, (B, C)),
                             "scale": (0.2, 0.05, (C,)), "w_pre": (1.0, 0.2, (C,)), "b_pre": (0.0, 0.1, (C,))}.items():
        t = torch.from_numpy(mid + dev * rng.standard_normal(s)).to(DT[dtype])
        prm[k] = None if k in absent else (t, t.double().numpy())
    return c, prm
