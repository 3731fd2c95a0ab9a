"""The block operators' float64 definitions (oracle/block.py) against published vectors and
differences, and the refusals of their entry points, without a GPU."""

import ctypes

import numpy as np
import pytest

import spectral_convolution_amd as fno
from oracle import block as ref
from spectral_convolution_amd import _lib

OK, INVALID, UNSUPPORTED = 0, 1, 2


# ------------------------------------------------------------------- oracle

def test_philox_known_answers():
    """The generator's published test vectors (counter and key of zeros, of ones, and digits of pi)."""
    hexes = lambda w: " ".join(f"{int(v):08x}" for v in np.ravel(w))  # noqa: E731
    ones = (1 << 64) - 1
    assert hexes(ref.philox(0, 0, 0)) == "6627e8d5 e169c58d bc57ac4c 9b00dbd8"
    assert hexes(ref.philox(ones, ones, ones)) == "408f276d 41c83b0e a20bc7c6 6d5451fd"
    assert hexes(ref.philox(0x85a308d3243f6a88, 0x0370734413198a2e, 0x299f31d0a4093822)) == \
        "d16cfe09 94fdcceb 5001e420 24126ea1"


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.1, 0.5, 0.9, 1.0])
def test_kept_share(p):
    n = 1 << 17
    kept = ref.kept_units(n, p, 12345, 7).mean()
    q = 1 - ref.drop_threshold(p) / 65536
    assert abs(kept - q) <= 5 * np.sqrt(q * (1 - q) / n)
    f = ref.drop_factor(1, 1, n, False, p, 12345, 7)
    assert p == 1.0 or abs(f.mean() - 1) <= 5 * np.sqrt((1 / q - 1) / n) + 1e-12


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("last", [False, True])
def test_group_norm_gradients_against_differences(kind, last):
    rng = np.random.default_rng(kind)
    B, C, P, G, eps = 2, 6, 5, 3, 1e-3
    x = rng.standard_normal((B, P, C) if last else (B, C, P))
    w, b = 1 + 0.3 * rng.standard_normal(C), 0.2 * rng.standard_normal(C)
    gy = rng.standard_normal(x.shape)
    f = ref.drop_factor(B, C, P, last, 0.3, 5)
    loss = lambda x, w, b: (ref.group_norm(x, G, eps, w, b, kind, last, f)[0] * gy).sum()  # noqa: E731
    got, _ = ref.group_norm_backward(x, G, eps, w, b, kind, last, gy, f)
    for i, t in enumerate((x, w, b)):
        for j in range(t.size):
            d = np.zeros(t.size)
            d[j] = 1e-5
            args = [[x, w, b], [x, w, b]]
            args[0][i], args[1][i] = t + d.reshape(t.shape), t - d.reshape(t.shape)
            diff = (loss(*args[0]) - loss(*args[1])) / 2e-5
            assert abs(diff - got[i].ravel()[j]) < 1e-7 * max(1, abs(diff))


# ----------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def _mem(n=1 << 16):
    """n bytes of host memory at a multiple of 256 (nothing reads it: the calls are refused)."""
    buf = ctypes.create_string_buffer(n + 256)
    a = ctypes.addressof(buf)
    _mem.keep.append(buf)
    return a + -a % 256


_mem.keep = []


def _gn(L, fwd=True, drop=None, **k):
    a = dict(groups=2, act=0, last=0, eps=1e-5, w=_mem(), b=_mem(), x=_mem(), y=_mem(), stats=_mem(), ws=_mem(), gy=_mem(),
             gx=_mem(), gw=_mem(), gb=_mem(), B=2, C=4, P=16, dt=0)
    a.update(k)
    p = _lib.GroupNormParamsStruct(a["groups"], a["act"], a["last"], a["eps"], a["w"], a["b"])
    p = None if a.get("params", 1) is None else ctypes.byref(p)
    d = None if drop is None else ctypes.byref(drop)
    if fwd:
        return L.fno_group_norm(p, d, a["x"], a["y"], a["stats"], a["ws"], a["B"], a["C"], a["P"], a["dt"], None)
    return L.fno_group_norm_backward(p, d, a["x"], a["stats"], a["gy"], a["gx"], a["gw"], a["gb"], a["ws"], a["B"], a["C"],
                                     a["P"], a["dt"], None)


NAN = float("nan")


@pytest.mark.parametrize("fwd", [True, False])
@pytest.mark.parametrize("k,expect", [
    (dict(groups=3), INVALID), (dict(groups=0), INVALID), (dict(groups=-2), INVALID), (dict(act=3), INVALID),
    (dict(act=-1), INVALID), (dict(last=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=NAN), INVALID),
    (dict(eps=-1e-5), INVALID), (dict(eps=1e-45), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID),
    (dict(P=0), INVALID), (dict(dt=3), INVALID), (dict(x=None), INVALID), (dict(ws=None), INVALID),
    (dict(params=None), INVALID), (dict(C=8194), UNSUPPORTED), (dict(P=(1 << 27) + 1), UNSUPPORTED),
    (dict(B=1 << 30, C=4, groups=4), UNSUPPORTED), (dict(B=1 << 20, C=8192, P=1 << 20), UNSUPPORTED)])
def test_group_norm_refuses(L, fwd, k, expect):
    assert _gn(L, fwd, **k) == expect


def test_group_norm_refuses_pointers(L):
    m = _mem()
    assert _gn(L, x=m, y=m) == INVALID
    assert _gn(L, x=m, y=m + 16) == INVALID
    assert _gn(L, x=m + 4) == INVALID
    assert _gn(L, y=None) == INVALID
    assert _gn(L, stats=m + 4) == INVALID
    assert _gn(L, ws=m + 8) == INVALID
    assert _gn(L, w=m + 2) == INVALID
    assert _gn(L, False, stats=None) == INVALID
    assert _gn(L, False, gy=None) == INVALID
    assert _gn(L, False, gx=None, gw=None, gb=None) == INVALID
    assert _gn(L, False, w=None) == INVALID
    assert _gn(L, False, b=None) == INVALID
    assert _gn(L, False, x=m, gx=m) == INVALID
    assert _gn(L, False, gw=m, gb=m) == INVALID


@pytest.mark.parametrize("drop", [(NAN, 0), (-0.1, 0), (1.1, 0), (0.5, 3), (0.5, -1)])
def test_dropout_refuses(L, drop):
    d = _lib.DropoutStruct(drop[0], drop[1], 1, 2, None)
    assert _gn(L, drop=d) == INVALID and _gn(L, False, drop=d) == INVALID
    assert L.fno_dropout_residual(ctypes.byref(d), None, _mem(), _mem(), 2, 4, 16, 0, 0, None) == INVALID


def test_dropout_residual_refuses(L):
    d = ctypes.byref(_lib.DropoutStruct(0.5, 0, 1, 2, None))
    m, o = _mem(), _mem()
    f = L.fno_dropout_residual
    assert f(None, None, m, o, 2, 4, 16, 0, 0, None) == INVALID
    assert f(d, None, None, o, 2, 4, 16, 0, 0, None) == INVALID
    assert f(d, None, m, None, 2, 4, 16, 0, 0, None) == INVALID
    assert f(d, None, m, m, 2, 4, 16, 0, 0, None) == INVALID
    assert f(d, o, m, o, 2, 4, 16, 0, 0, None) == INVALID
    assert f(d, None, m + 8, o, 2, 4, 16, 0, 0, None) == INVALID
    for B, C, P, last, dt in ((0, 4, 16, 0, 0), (2, 0, 16, 0, 0), (2, 4, 0, 0, 0), (2, 4, 16, 2, 0), (2, 4, 16, 0, 5)):
        assert f(d, None, m, o, B, C, P, last, dt, None) == INVALID
    assert f(d, None, m, o, 1 << 20, 1 << 20, 2, 0, 0, None) == UNSUPPORTED
    assert f(d, None, m, o, 1, 1, (1 << 31) + 1, 0, 0, None) == UNSUPPORTED
    odd = ctypes.byref(_lib.DropoutStruct(0.5, 0, 1, 2, m + 4))
    assert f(odd, None, m, o, 2, 4, 16, 0, 0, None) == INVALID
    over = ctypes.byref(_lib.DropoutStruct(0.5, 0, 1, 2, o))  # the step's memory is an output
    assert f(over, None, m, o, 2, 4, 16, 0, 0, None) == INVALID


def test_a_dropout_does_not_change():
    """Its backward would draw another mask, or the change would be lost."""
    import copy
    d = fno.Dropout(0.25, 3, 7, unit="channel")
    for name in ("p", "seed", "offset", "unit", "step"):
        with pytest.raises(AttributeError):
            setattr(d, name, 1)
    e = copy.deepcopy(d)
    assert (e.p, e.seed, e.offset, e.unit, e.step) == (0.25, 3, 7, "channel", None)
    assert (e._s.p, e._s.unit, e._s.seed, e._s.offset) == (0.25, 1, 3, 7)


def test_binding_refuses():
    import torch
    for bad in (-0.1, 1.5, NAN):
        with pytest.raises(ValueError):
            fno.Dropout(bad, 1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=1, offset=-1), dict(seed=1, unit="row"),
               dict(seed=1, step=torch.zeros(2, dtype=torch.int64)), dict(seed=1, step=torch.zeros(1)), dict(seed=1, step=3)):
        with pytest.raises(ValueError):
            fno.Dropout(0.5, **kw)
    with pytest.raises(ValueError):
        fno.GroupNormParams(2, act=3)
    with pytest.raises(ValueError):
        fno.GroupNormParams(0)
    x = torch.zeros(2, 4, 16)
    d = fno.Dropout(0.5, 1)
    with pytest.raises(ValueError):  # on the host
        fno.fno_dropout_residual(d, None, x, torch.zeros_like(x))
    with pytest.raises(TypeError):
        fno.fno_dropout_residual(None, None, x, torch.zeros_like(x))
    with pytest.raises(ValueError):
        fno.group_norm(x, fno.GroupNormParams(2))
    with pytest.raises(ValueError):
        fno.fno_dropout_residual(d, None, x, torch.zeros(2, 4, 15))
    with pytest.raises(ValueError):
        fno.fno_dropout_residual(d, None, x[..., ::2], x[..., ::2])
    with pytest.raises(ValueError):
        fno.fno_dropout_residual(d, None, x.double(), x.double())
    with pytest.raises(ValueError):
        fno.fno_group_norm_workspace_empty(x[0, 0], 2)


def test_mx4_definition():
    """Exact values keep, ties go to the even code, the cut is at 6, the error is as documented."""
    v = np.array([[0, 0.5, 1, 1.5, 2, 3, 4, 6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.99, -0.0, -5.1] + [0.0] * 14])
    q, s = ref.mx4(v)
    assert s[0, 0] == 127
    assert list(q[0, 0, :18]) == [0, 1, 2, 3, 4, 5, 6, 7, 0, 2, 2, 4, 4, 6, 6, 7, 8, 15]
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(2 * rng.standard_normal((50, 96)))
    got = ref.mx4_trip(x)
    M = abs(x).reshape(50, 3, 32).max(-1).repeat(32, -1).reshape(50, 96)
    assert (abs(got - x) <= M / 4).all()
    unit = 2.0 ** (np.floor(np.log2(M)) - 2)  # half the widest step between values below the cut
    assert (abs(got - x) <= unit)[abs(x) <= 6 * unit].all()
    assert np.array_equal(ref.mx4_trip(got), got)


def test_mx4_refuses(L):
    n = ctypes.c_size_t()
    m, o, z = _mem(), _mem(), _mem()
    for B, C, P, st in ((0, 4, 4, INVALID), (2, 0, 4, INVALID), (2, 4, 0, INVALID), (2, 65537, 1, UNSUPPORTED),
                        (2, 32, (1 << 30) + 1, UNSUPPORTED), (1 << 20, 65536, 1 << 6, UNSUPPORTED)):
        assert L.fno_mx4_bytes(B, C, P, ctypes.byref(n)) == st
        assert L.fno_mx4_pack(m, o, B, C, P, 0, None) == st
        assert L.fno_mx4_unpack(m, o, B, C, P, 0, None) == st
        assert L.fno_channel_mix_mx4(m, o, None, None, z, B, C, 4, P, 0, 0, None) == st
        assert L.fno_channel_mix_mx4(m, o, None, None, z, B, 4, C, P, 0, 0, None) == st
    assert L.fno_mx4_bytes(2, 4, 4, None) == INVALID
    for f in (L.fno_mx4_pack, L.fno_mx4_unpack):
        assert f(None, o, 2, 4, 4, 0, None) == INVALID
        assert f(m, None, 2, 4, 4, 0, None) == INVALID
        assert f(m, m, 2, 4, 4, 0, None) == INVALID
        assert f(m, o, 2, 4, 4, 7, None) == INVALID
        assert f(m + 8, o, 2, 4, 4, 0, None) == INVALID
        assert f(m, o + 8, 2, 4, 4, 0, None) == INVALID
    assert L.fno_mx4_pack(m, o + 16, 2, 4, 4, 0, None) == INVALID  # packed: 256 bytes
    f = L.fno_channel_mix_mx4
    assert f(None, o, None, None, z, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, None, None, None, z, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, None, None, None, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, None, None, z, 2, 4, 4, 4, 2, 0, None) == INVALID
    assert f(m, o, None, None, z, 2, 4, 4, 4, 0, 3, None) == INVALID
    assert f(m + 16, o, None, None, z, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, z, None, z, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, None, z, z, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, None, None, m, 2, 4, 4, 4, 0, 0, None) == INVALID
    assert f(m, o, z + 2, None, _mem(), 2, 4, 4, 4, 0, 0, None) == INVALID


@pytest.mark.parametrize("call", [
    lambda: fno.fno_mx4_bytes((1 << 32) + 2, 4), lambda: fno.fno_mx4_bytes(2, (1 << 32) + 4),
    lambda: fno.fno_mx4_bytes(2, 4, (1 << 64) + 4),
    lambda: fno.fno_group_norm_workspace_bytes((1 << 32) + 2, 4, 16, 2),
    lambda: fno.fno_group_norm_workspace_bytes(2, (1 << 32) + 4, 16, 2),
    lambda: fno.fno_group_norm_workspace_bytes(2, 4, (1 << 64) + 16, 2),
    lambda: fno.fno_group_norm_workspace_bytes(2, 4, 16, (1 << 32) + 2),
])
def test_sizes_past_the_abis_integers(call):
    with pytest.raises(ValueError, match="range"):
        call()
