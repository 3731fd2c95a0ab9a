"""The fp32 training kernels' GELU and derivative, evaluated step by step in
float32 the way the kernels do, against the normal distribution in float64.

Bounds: the tail q = 1 - Phi(|v|) is at most 1/2 and passes through about ten
roundings of 2^-24, two of them (v^2 and its product) inside the exponential, where they
count v^2 / 2 e^(-v^2 / 2) <= 0.37 each: 8 2^-24 with the fit's 1e-8 is more than all
of them at their worst. GELU takes |v| q, the derivative q and v phi(v) <= 0.25."""

import math
import os
import re

import numpy as np
from scipy.special import ndtr

F = np.float32
STEP = 2.0 ** -24
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _coefficients():
    src = open(os.path.join(ROOT, "spectral_convolution_amd", "csrc", "gelu.hpp")).read()
    body = src[src.index("float normal_tail("):src.index("float normal_bell(")]
    first = re.search(r"float p = fmaf\(([-\d.e]+)f, t, ([-\d.e]+)f\)", body)
    rest = re.findall(r"p = fmaf\(p, t, ([-\d.e]+)f\)", body)
    slope = re.search(r"rcpf\(fmaf\(([-\d.e]+)f, a", body).group(1)
    return float(slope), [float(first.group(1)), float(first.group(2))] + [float(c) for c in rest]


def _fma(a, b, c):
    return (a.astype(np.float64) * b.astype(np.float64) + np.float64(c)).astype(F)


def _bell_and_tail(v):
    k, c = _coefficients()
    assert len(c) == 6
    e = np.exp2(((v * v).astype(F) * F(-0.72134752044448170)).astype(F).astype(np.float64)).astype(F)
    t = (F(1) / _fma(F(k), np.abs(v), 1.0)).astype(F)
    p = np.full_like(v, F(c[0]))
    for x in c[1:]:
        p = _fma(p, t, F(x))
    return e, ((p * t).astype(F) * e).astype(F)


def _values():
    return np.concatenate([np.linspace(-12, 12, 200001), [0.0, 1e-30, -1e-30, 50.0, -50.0, 1e30, -1e30]]).astype(F)


def test_tail():
    v = _values()
    with np.errstate(over="ignore"):
        _, q = _bell_and_tail(v)
    assert (abs(q - ndtr(-abs(v.astype(np.float64)))) <= 8 * STEP).all()


def test_gelu():
    v = _values()
    with np.errstate(over="ignore"):
        _, q = _bell_and_tail(v)
    g = _fma(-np.minimum(abs(v), F(100)), q, np.maximum(v, F(0)).astype(np.float64))
    ref = v.astype(np.float64) * ndtr(v.astype(np.float64))
    a = abs(v.astype(np.float64))
    assert (abs(g - ref) <= 8 * STEP * np.minimum(a, 8.0) + STEP * a).all()
    assert g[v == F(1e30)] == F(1e30) and g[v == F(-1e30)] == 0


def test_derivative():
    v = _values()
    with np.errstate(over="ignore"):
        e, q = _bell_and_tail(v)
    s = _fma((np.clip(v, F(-100), F(100)) * F(0.39894228040143268)).astype(F), e,
             np.where(v >= 0, (F(1) - q).astype(F), q).astype(np.float64))
    d = v.astype(np.float64)
    with np.errstate(over="ignore"):
        ref = ndtr(d) + d * np.exp(-0.5 * d * d) / math.sqrt(2 * math.pi)
    assert (abs(s - ref) <= 12 * STEP).all()
