"""The training operators' definitions and their refusals, without a GPU: the
float64 oracle against differences and against automatic differentiation, and
the C ABI's and the binding's checks of their arguments (which run before any
HIP call)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import training as ref
from spectral_convolution_amd import _lib
from training_util import LOW, norm_case

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


# ------------------------------------------------------------- the oracle

@pytest.mark.parametrize("low", [-126, -24])
def test_checkpoint_error_bound(low):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, 95)) * np.exp2(rng.integers(-30, 12, (6, 1)))
    y = ref.round_trip(x, low)
    for r in range(6):
        for k in range(0, 95, 32):
            b, g = x[r, k:k + 32], y[r, k:k + 32]
            big = abs(b).max()
            step = 2.0 ** max(math.floor(math.log2(big)) - 6, low)
            assert (abs(g - b) <= step / 2 + (abs(b) > 127 * step) * step / 2).all()
    assert (ref.round_trip(y, low) == y).all()  # what was kept is kept again


def test_checkpoint_of_a_power_of_two_and_of_poison():
    x = np.zeros((3, 32))
    x[0, 5] = 64.0
    x[1, 7] = np.inf
    x[2, 9] = np.nan
    q, e = ref.checkpoint(x, -126)
    assert e[0, 0] == 0 and q[0, 5] == 64 and e[1, 0] == e[2, 0] == 127
    v = ref.checkpoint_values(q, e, 32)
    assert (v[0] == x[0]).all() and np.isnan(v[1:]).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("P", [None, 5])
def test_norm_gradients_against_differences_and_autograd(kind, P):
    c, prm = norm_case("f32", 2, 6, P, seed=4)
    p = {k: v[1] for k, v in prm.items()}
    x, v, gy, gu = (c[k][1] for k in ("x", "v", "gy", "gu"))

    def loss(p, x, v):
        y, u = ref.norm_residual(p, kind, 1e-5, x, v)
        return (y * gy).sum() + (u * gu).sum()

    g = ref.norm_residual_backward(p, kind, 1e-5, x, v, gy, gu)
    rng = np.random.default_rng(5)
    h = 1e-6
    for name, got in (("x", g["gx"][0]), ("v", g["gv"][0])):
        d = rng.standard_normal(x.shape)
        lo, hi = ({"x": x, "v": v, name: {"x": x, "v": v}[name] + s * h * d} for s in (-1, 1))
        diff = (loss(p, hi["x"], hi["v"]) - loss(p, lo["x"], lo["v"])) / (2 * h)
        assert abs(diff - (got * d).sum()) <= 1e-7 * max(1, abs(diff))
    for k in p:
        d = rng.standard_normal(p[k].shape)
        diff = (loss({**p, k: p[k] + h * d}, x, v) - loss({**p, k: p[k] - h * d}, x, v)) / (2 * h)
        assert abs(diff - (g[k][0] * d).sum()) <= 1e-7 * max(1, abs(diff)), k


@pytest.mark.parametrize("act", [0, 1])
def test_mix_gradients_against_autograd(act):
    rng = np.random.default_rng(6)
    x, A, b, add, gy = (rng.standard_normal(s) for s in ((2, 3, 7), (4, 3), (4,), (2, 4, 7), (2, 4, 7)))
    leaves = [torch.from_numpy(t).requires_grad_() for t in (x, A, b, add)]
    z = torch.matmul(leaves[1], leaves[0]) + leaves[2][:, None] + leaves[3]
    out = z * torch.special.ndtr(z) if act else z
    want = torch.autograd.grad(out, leaves, torch.from_numpy(gy))
    got, _ = ref.channel_mix_backward(x, A, b, add, gy, act)
    assert np.allclose(ref.channel_mix(x, A, b, add, act), out.detach().numpy(), rtol=1e-13, atol=1e-13)
    for g, w in zip(got, want):
        assert np.allclose(g, w.numpy(), rtol=1e-12, atol=1e-12)


# --------------------------------------------------------------- refusals

def _buf(n, align=256):
    b = ctypes.create_string_buffer(n + align)
    a = (ctypes.addressof(b) + align - 1) // align * align
    return b, a


def test_checkpoint_sizes(L):
    n = ctypes.c_size_t(7)
    for rows, length in ((1, 1), (3, 32), (5, 33), (96, 3721), (1, 1 << 31)):
        nb = -(-length // 32)
        assert L.fno_checkpoint_bytes(rows, length, ctypes.byref(n)) == OK
        assert n.value == -(-rows * nb * 32 // 256) * 256 + -(-rows * nb // 256) * 256
    n.value = 7
    assert L.fno_checkpoint_bytes(0, 4, ctypes.byref(n)) == INVALID
    assert L.fno_checkpoint_bytes(4, 0, ctypes.byref(n)) == INVALID
    assert L.fno_checkpoint_bytes(4, 4, None) == INVALID
    assert L.fno_checkpoint_bytes(1, (1 << 31) + 1, ctypes.byref(n)) == UNSUPPORTED
    assert L.fno_checkpoint_bytes(1 << 40, 32, ctypes.byref(n)) == UNSUPPORTED
    assert n.value == 7


def test_checkpoint_refusals(L):
    keep, a = _buf(8192)
    x, saved = a, a + 4096
    for f in (lambda x, s, *r: L.fno_checkpoint_pack(x, s, *r, None),
              lambda x, s, *r: L.fno_checkpoint_unpack(s, x, *r, None)):
        assert f(None, saved, 2, 40, 0) == INVALID
        assert f(x, None, 2, 40, 0) == INVALID
        assert f(x, saved, 0, 40, 0) == INVALID
        assert f(x, saved, 2, -1, 0) == INVALID
        assert f(x, saved, 2, 40, 3) == INVALID
        assert f(x + 2, saved, 2, 40, 1) == INVALID         # field off 16 bytes
        assert f(x, saved + 64, 2, 40, 0) == INVALID        # buffer off 256 bytes
        assert f(x, x + 256, 2, 40, 0) == INVALID           # overlap: the field is 320 bytes
        assert f(x, saved, 1, (1 << 31) + 8, 0) == UNSUPPORTED


def _norm_call(L, **change):
    keep, a = _buf(1 << 16)
    C = change.pop("C", 4)
    d = dict(kind=0, eps=1e-5, w_post=a, b_post=a + 64, gate=a + 128, scale=a + 192, w_pre=a + 256, b_pre=a + 320,
             x=a + 4096, v=a + 8192, y=a + 12288, u=a + 16384, saved=a + 20480, B=2, P=16, dtype=0)
    given = {k: change.pop(k) for k in list(change) if k in d}
    d.update({k: a + v[1] if isinstance(v, tuple) else v for k, v in given.items()})
    assert not change
    st = _lib.NormParamsStruct(*(d[k] for k in ("kind", "eps", "w_post", "b_post", "gate", "scale", "w_pre", "b_pre")))
    ref_ = ctypes.byref(st) if d["x"] != "no params" else None
    x = None if d["x"] == "no params" else d["x"]
    tail = (d["B"], C, d["P"], d["dtype"], None)
    return (L.fno_norm_residual(ref_, x, d["v"], d["y"], d["u"], *tail),
            L.fno_norm_residual_save(ref_, x, d["v"], d["y"], d["u"], d["saved"], *tail))


@pytest.mark.parametrize("change,expect", [
    (dict(x="no params"), INVALID), (dict(x=None), INVALID), (dict(v=None), INVALID), (dict(y=None), INVALID),
    (dict(kind=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(eps=1e-42), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID),
    (dict(P=0), INVALID), (dict(dtype=3), INVALID), (dict(x=("a", 4098), dtype=1), INVALID),
    (dict(gate=("a", 129), dtype=1), INVALID),
    (dict(y=("a", 4096 + 256)), INVALID),                      # y overlaps x
    (dict(u=("a", 12288)), INVALID),                           # u is y
    (dict(y=("a", 64)), INVALID),                              # y overlaps a parameter
    (dict(C=513), UNSUPPORTED), (dict(C=8193, P=1), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(B=60000, C=512, P=1 << 20), UNSUPPORTED),
])
def test_norm_forward_refusals(L, change, expect):
    assert _norm_call(L, **dict(change)) == (expect, expect)


def test_norm_save_refuses_its_buffer(L):
    assert _norm_call(L, x=None, saved=None)[1] == INVALID
    keep, a = _buf(1 << 16)
    st = _lib.NormParamsStruct(0, 1e-5)
    f = lambda s: L.fno_norm_residual_save(ctypes.byref(st), a, a + 4096, a + 8192, None, s, 2, 4, 16, 0, None)  # noqa: E731
    assert f(None) == INVALID and f(a + 20480 + 128) == INVALID and f(a) == INVALID


def test_norm_backward_refusals(L):
    keep, a = _buf(1 << 17)
    full = dict(w_post=a, b_post=a + 64, gate=a + 128, scale=a + 192, w_pre=a + 256, b_pre=a + 320)
    x, v, gy, gu, gx, gv, ws, saved = (a + 4096 * (1 + i) for i in range(8))
    gr = {k: a + 36864 + 64 * i for i, k in enumerate(full)}

    def call(prm=full, grads=gr, x=x, v=v, gy=gy, gu=gu, gx=gx, gv=gv, ws=ws, saved=saved, C=4, dtype=0):
        p = _lib.NormParamsStruct(1, 1e-5, **prm)
        g = None if grads is None else ctypes.byref(_lib.NormGradsStruct(**grads))
        one = L.fno_norm_residual_backward(ctypes.byref(p), x, v, gy, gu, gx, gv, g, ws, 2, C, 16, dtype, None)
        two = L.fno_norm_residual_backward_saved(ctypes.byref(p), saved, gy, gu, gx, gv, g, ws, 2, C, 16, dtype, None)
        return one, two

    bad = (INVALID, INVALID)
    assert call(gy=None) == bad and call(ws=None) == bad and call(dtype=4) == bad
    assert call(x=None)[0] == INVALID and call(v=None)[0] == INVALID and call(saved=None)[1] == INVALID
    assert call(gx=None, gv=None, grads=None) == bad                     # nothing wanted
    assert call(prm={**full, "gate": None}) == bad                       # gradient of an absent parameter
    assert call(gu=None) == bad                                          # w_pre's gradient without gu
    assert call(gx=gy) == bad and call(gx=gv) == bad and call(gv=ws) == bad
    assert call(grads={**gr, "gate": full["gate"]}) == bad               # a gradient over its parameter
    assert call(gx=gx + 8) == bad and call(ws=ws + 8) == bad
    assert call(saved=saved + 16)[1] == INVALID
    assert call(C=513) == (UNSUPPORTED, UNSUPPORTED)


def test_norm_sizes(L):
    n = ctypes.c_size_t()
    assert L.fno_norm_residual_saved_bytes(3, 5, 70, ctypes.byref(n)) == OK
    assert n.value == 2 * (-(-15 * 96 // 256) * 256 + 256)
    assert L.fno_norm_residual_saved_bytes(3, 70, 1, ctypes.byref(n)) == OK
    assert n.value == 2 * (-(-3 * 96 // 256) * 256 + 256)
    assert L.fno_norm_residual_saved_bytes(3, 5, 70, None) == INVALID
    assert L.fno_norm_residual_saved_bytes(0, 5, 70, ctypes.byref(n)) == INVALID
    assert L.fno_norm_residual_workspace_bytes(3, 5, 70, 7, ctypes.byref(n)) == INVALID
    assert L.fno_norm_residual_workspace_bytes(3, 5, 70, 0, ctypes.byref(n)) == OK and n.value > 0


def test_binding_refuses_host_tensors_and_mismatches():
    x = torch.zeros(2, 4, 16)
    prm = fno.NormParams("rms", 1e-5)
    with pytest.raises(ValueError, match="shape"):
        fno.fno_norm_residual(prm, x, x[:, :3], x, x)
    with pytest.raises(ValueError, match="dtype"):
        fno.fno_norm_residual(prm, x, x.half(), x, x)
    with pytest.raises(ValueError, match="gate shape"):
        fno.fno_norm_residual(fno.NormParams("rms", 1e-5, gate=torch.zeros(4)), x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        fno.fno_norm_residual(prm, x, x, x, x)
    with pytest.raises(ValueError, match="kind"):
        fno.NormParams("batch", 1e-5)
    with pytest.raises(ValueError, match="holds"):
        fno.fno_checkpoint_pack(x, torch.zeros(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dtype"):
        fno.fno_checkpoint_pack(x.double(), torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(TypeError):
        fno.fno_norm_residual_backward(prm, x, None, x, x, x, x, None, None)


# ------------------------------------------------------------- channel mix

def test_mix_sizes(L):
    n = ctypes.c_size_t(7)
    x, add = -(-6 * 128 // 256) * 256 + 256, -(-10 * 128 // 256) * 256 + 256
    for act, has_add, want in ((0, 0, x), (0, 1, x), (1, 0, x), (1, 1, x + add)):
        assert L.fno_channel_mix_saved_bytes(2, 3, 5, 100, act, has_add, ctypes.byref(n)) == OK and n.value == want
    assert L.fno_channel_mix_saved_bytes(2, 3, 5, 100, 2, 0, ctypes.byref(n)) == INVALID
    assert L.fno_channel_mix_saved_bytes(2, 3, 5, 100, 1, 0, None) == INVALID
    assert L.fno_channel_mix_saved_bytes(2, 129, 5, 100, 1, 0, ctypes.byref(n)) == UNSUPPORTED
    assert L.fno_channel_mix_workspace_bytes(2, 3, 129, 100, 0, ctypes.byref(n)) == UNSUPPORTED
    assert L.fno_channel_mix_workspace_bytes(2, 3, 5, 0, 0, ctypes.byref(n)) == INVALID
    assert L.fno_channel_mix_workspace_bytes(2, 3, 5, 100, 0, ctypes.byref(n)) == OK and 0 < n.value


def test_mix_refusals(L):
    keep, a = _buf(1 << 17)
    at = {k: a + 8192 * i for i, k in enumerate(("x", "A", "bias", "add", "y", "saved", "gy", "gx", "gA", "gbias",
                                                 "gadd", "ws"))}

    def fwd(I=3, O=5, P=100, B=2, act=1, dtype=0, **kw):
        d = {**at, **kw}
        return L.fno_channel_mix_save(d["x"], d["A"], d["bias"], d["add"], d["y"], d["saved"], B, I, O, P, act, dtype,
                                      None)

    def bwd(I=3, O=5, P=100, B=2, act=1, has_add=1, dtype=0, **kw):
        d = {**at, **kw}
        return L.fno_channel_mix_backward_saved(d["saved"], d["A"], d["bias"], d["gy"], d["gx"], d["gA"], d["gbias"],
                                                d["gadd"], d["ws"], B, I, O, P, act, has_add, dtype, None)

    for k in ("x", "A", "y", "saved"):
        assert fwd(**{k: None}) == INVALID
    for k in ("gy", "A", "saved", "ws"):
        assert bwd(**{k: None}) == INVALID
    for f in (fwd, bwd):
        for bad in (dict(I=0), dict(O=0), dict(P=0), dict(B=0), dict(act=2), dict(dtype=3)):
            assert f(**bad) == INVALID
        for far in (dict(I=129), dict(O=129), dict(P=(1 << 31) + 1)):
            assert f(**far) == UNSUPPORTED
        assert f(saved=at["saved"] + 128) == INVALID and f(A=at["A"] + 1) == INVALID
    assert fwd(y=at["x"]) == INVALID and fwd(y=at["add"]) == INVALID and fwd(saved=at["x"]) == INVALID
    assert fwd(x=at["x"] + 8) == INVALID
    assert bwd(gx=None, gA=None, gbias=None, gadd=None) == INVALID
    assert bwd(has_add=0) == INVALID                                     # gadd without an add input
    assert bwd(has_add=2) == INVALID
    assert bwd(gx=at["gy"]) == INVALID and bwd(gadd=at["gy"]) == INVALID and bwd(gA=at["A"]) == INVALID
    assert bwd(ws=at["gx"]) == INVALID and bwd(ws=at["ws"] + 4) == INVALID


def test_mix_binding_mismatches():
    x, A = torch.zeros(2, 3, 40), torch.zeros(5, 3)
    y, big = torch.zeros(2, 5, 40), torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="y shape"):
        fno.fno_channel_mix_save(x, A, None, None, torch.zeros(2, 5, 41), big)
    with pytest.raises(ValueError, match="A shape"):
        fno.fno_channel_mix_save(x, A.t(), None, None, y, big)
    with pytest.raises(ValueError, match="add dtype"):
        fno.fno_channel_mix_save(x, A, None, y.half(), y, big)
    with pytest.raises(ValueError, match="does not map"):
        fno.fno_channel_mix_backward_saved(big, A.t(), None, y, x, None, None, None, None)
    with pytest.raises(ValueError, match="saved holds"):
        fno.fno_channel_mix_backward_saved(big[:8], A, None, y, x, None, None, None, None)
    with pytest.raises(TypeError, match="workspace"):
        fno.fno_channel_mix_backward_saved(big[-big.data_ptr() % 256:], A, None, y, x, A, None, None, None)


# ------------------------------------------------- differentiable functions

def test_differentiable_functions_refuse():
    x, A = torch.zeros(2, 3, 5), torch.zeros(4, 3)
    with pytest.raises(ValueError, match="on the GPU"):
        fno.channel_mix(x, A)
    with pytest.raises(ValueError, match="c_out"):
        fno.channel_mix(x, torch.zeros(4))
    prm = fno.NormParams("rms", 1e-5)
    with pytest.raises(ValueError, match="keep"):
        fno.norm_residual(x, x, prm, keep="4bit")
    with pytest.raises(ValueError, match="on the GPU"):
        fno.norm_residual(x, x, prm)


def test_example_data_is_the_heat_equations():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_conditioned_fno2d.py")
    spec = importlib.util.spec_from_file_location("train_conditioned_fno2d", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    a, tau, s = m.heat_batch(np.random.default_rng(1), 3, (16, 24))
    assert a.shape == s.shape == (3, 1, 16, 24) and (0 <= tau).all() and (tau < 1).all()
    assert np.allclose(a.mean((2, 3)), s.mean((2, 3)))
    # one mode by hand: 2 periods along the second axis
    k2 = (2 * math.pi * 2) ** 2
    fa, fs = np.fft.fft2(a)[..., 0, 2], np.fft.fft2(s)[..., 0, 2]
    assert np.allclose(fs[:, 0], fa[:, 0] * np.exp(-m.TAU * tau * k2))
