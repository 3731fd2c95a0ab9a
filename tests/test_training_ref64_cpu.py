"""tests/training_ref64.py against the oracle."""

import numpy as np
import pytest
import torch

import training_ref64 as r64
from oracle import training as ref
from training_util import norm_case

TINY = dict(rtol=1e-12, atol=1e-13)


def _t(a):
    return None if a is None else torch.from_numpy(np.asarray(a))


@pytest.mark.parametrize("low", [-126, -24])
def test_round_trip(low):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 75)) * np.exp2(rng.integers(-40, 12, (5, 3, 1)))
    x[0, 0] = 0
    x[1, 1, 3] = 4.0
    assert (r64.round_trip(_t(x), low).numpy() == ref.round_trip(x, low)).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("P", [None, 9])
@pytest.mark.parametrize("absent", [(), ("gate", "b_post"), ("scale", "w_post", "w_pre", "b_pre")])
@pytest.mark.parametrize("use_u", [True, False])
def test_norm(kind, P, absent, use_u):
    c, prm = norm_case("f32", 3, 7, P, seed=2, absent=absent)
    p = {k: None if t is None else t[1] for k, t in prm.items()}
    x, v, gy, gu = (c[k][1] for k in ("x", "v", "gy", "gu"))
    pt = {k: _t(t) for k, t in p.items()}
    for a, b in zip(r64.norm_residual(pt, kind, 1e-5, _t(x), _t(v)), ref.norm_residual(p, kind, 1e-5, x, v)):
        assert np.allclose(a.numpy(), b, **TINY)
    got = r64.norm_residual_backward(pt, kind, 1e-5, _t(x), _t(v), _t(gy), _t(gu) if use_u else None)
    want = ref.norm_residual_backward(p, kind, 1e-5, x, v, gy, gu if use_u else None)
    assert got.keys() == want.keys()
    for k in want:
        for a, b in zip(got[k], want[k]):
            assert np.allclose(a.numpy(), b, **TINY), k


@pytest.mark.parametrize("act", [0, 1])
def test_mix(act):
    rng = np.random.default_rng(3)
    x, A, b, add, gy = (rng.standard_normal(s) for s in ((2, 3, 7), (4, 3), (4,), (2, 4, 7), (2, 4, 7)))
    t = [_t(s) for s in (x, A, b, add)]
    assert np.allclose(r64.channel_mix(*t, act).numpy(), ref.channel_mix(x, A, b, add, act), **TINY)
    want, _ = ref.channel_mix_backward(x, A, b, add, gy, act)
    for g, w in zip(r64.channel_mix_backward(*t, _t(gy), act), want):
        assert np.allclose(g.numpy(), w, **TINY)
