"""GPU parity of the training operators around a block against their float64
definitions (oracle/training.py), at the sizes and values where they can go
wrong: rows of one value, rows that end inside a block or a tile, odd channel
counts, constant and empty-handed rows, poisoned values, absent parameters,
gradients that are not wanted, other streams and captured graphs."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import training as ref
from training_util import DT, LOW, NORM_NAMES, close, f64, norm_case, stored

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]
DEV = "cuda:0"


def dev(t):
    return None if t is None else t.to(DEV)


# ------------------------------------------------------------- checkpoints

def _parts(saved, rows, n):
    nb = -(-n // 32)
    off = -(-rows * nb * 32 // 256) * 256
    b = saved.cpu().view(torch.int8)
    return b[:rows * nb * 32].view(rows, -1).numpy(), b[off:off + rows * nb].view(rows, nb).numpy()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (7, 1), (3, 31), (2, 32), (5, 33), (1, 255), (9, 1000), (96, 3721),
                                    (2, 8191), (300, 40), (4, 4096), (1, 100003)])
def test_checkpoint(dtype, rows, n):
    rng = np.random.default_rng(rows * 1000 + n)
    x, x64 = stored(rng, (rows, n), dtype, spread=True)
    saved = torch.full((fno.fno_checkpoint_bytes(rows, n),), 77, dtype=torch.uint8, device=DEV)
    y = torch.full((rows, n), 3.0, dtype=DT[dtype], device=DEV)
    fno.fno_checkpoint_pack(dev(x), saved)
    fno.fno_checkpoint_unpack(saved, y)
    q, e = ref.checkpoint(x64, LOW[dtype])
    gq, ge = _parts(saved, rows, n)
    assert (gq == q).all() and (ge == e).all()
    assert (f64(y) == ref.checkpoint_values(q, e, n)).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_checkpoint_of_extreme_values(dtype):
    fi = torch.finfo(DT[dtype])
    tiny = 2.0 ** -24 if dtype == "f16" else (2.0 ** -149 if dtype == "f32" else 2.0 ** -133)
    rows = [[0.0] * 40, [-0.0] * 40, [fi.max] * 40, [fi.min, fi.max, fi.tiny] + [1.0] * 37, [tiny] * 40,
            [fi.tiny, -tiny, 3 * tiny] + [0.0] * 37, [fi.tiny] * 40,
            [2.0 ** -6 * (127.5 + 1e-9)] + [1.0] * 39, [2.0 - float(fi.eps)] * 40, [-2.0] * 40,
            [1.5 * 2.0 ** -6, 2.5 * 2.0 ** -6, 1.0, -1.5 * 2.0 ** -6, -2.5 * 2.0 ** -6] + [0.0] * 35]
    x = torch.tensor(rows, dtype=torch.float64).to(DT[dtype])
    x64 = x.double().numpy()
    saved, y = fno.fno_checkpoint_empty(dev(x)), torch.empty_like(dev(x))
    fno.fno_checkpoint_pack(dev(x), saved)
    fno.fno_checkpoint_unpack(saved, y)
    assert (f64(y) == ref.round_trip(x64, LOW[dtype])).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_checkpoint_of_poisoned_blocks(dtype):
    x = torch.ones(4, 100)
    x[0, 5], x[1, 40], x[2, 99] = float("nan"), float("inf"), -float("inf")
    x = x.to(DT[dtype])
    saved, y = fno.fno_checkpoint_empty(dev(x)), torch.empty_like(dev(x))
    fno.fno_checkpoint_pack(dev(x), saved)
    fno.fno_checkpoint_unpack(saved, y)
    bad = np.zeros((4, 100), bool)
    bad[0, :32] = bad[1, 32:64] = bad[2, 96:] = True
    got = f64(y)
    assert (np.isnan(got) == bad).all() and (got[~bad] == 1.0).all()


def test_checkpoint_keeps_what_it_kept():
    x, _ = stored(np.random.default_rng(2), (17, 333), "bf16", spread=True)
    x = dev(x)
    saved, y, again = fno.fno_checkpoint_empty(x), torch.empty_like(x), torch.empty_like(x)
    fno.fno_checkpoint_pack(x, saved)
    fno.fno_checkpoint_unpack(saved, y)
    fno.fno_checkpoint_pack(y, saved)
    fno.fno_checkpoint_unpack(saved, again)
    assert torch.equal(y, again)


# ------------------------------------------------------------------- norms

# (B, C, P): P None is the token layout
SHAPES = [(2, 4, 256), (1, 1, 2), (3, 7, 33), (2, 8, 64), (1, 13, 1000), (2, 16, 70), (3, 32, 31), (1, 33, 129),
          (2, 48, 3721), (1, 64, 512), (1, 65, 100), (2, 128, 65), (1, 200, 257), (1, 256, 64), (1, 257, 97),
          (1, 512, 40), (1, 1, None), (3, 5, None), (5, 64, None), (9, 257, None), (4, 500, None), (3, 512, None),
          (2, 1000, None), (6, 1024, None), (3, 1025, None), (2, 3001, None), (2, 4096, None), (1, 8191, None),
          (2, 8192, None), (1500, 40, None)]


def _params(prm):
    return {k: None if v is None else dev(v[0]) for k, v in prm.items()}


def _run(dtype, kind, c, prm, saved_form, eps=1e-5, want=NORM_NAMES, use_u=True, stream=None):
    x, v, gy, gu = (dev(c[k][0]) for k in ("x", "v", "gy", "gu"))
    p = _params(prm)
    N = fno.NormParams(kind, eps, **p)
    y = torch.full_like(x, 7.0)
    u = torch.full_like(x, 7.0) if use_u else None
    gx, gv = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    grads = {k: torch.full_like(p[k], 7.0) for k in want if p[k] is not None and (use_u or not k.endswith("_pre"))}
    ws = torch.full_like(fno.fno_norm_residual_workspace_empty(x), 255)
    if saved_form:
        kept = torch.full_like(fno.fno_norm_residual_saved_empty(x), 99)
        fno.fno_norm_residual_save(N, x, v, y, u, kept)
        fno.fno_norm_residual_backward_saved(N, kept, gy, gu if use_u else None, gx, gv, fno.NormGrads(**grads), ws)
    else:
        fno.fno_norm_residual(N, x, v, y, u)
        fno.fno_norm_residual_backward(N, x, v, gy, gu if use_u else None, gx, gv, fno.NormGrads(**grads), ws)
    return y, u, gx, gv, grads


def _check(dtype, kind, c, prm, saved_form, eps=1e-5, use_u=True, want=NORM_NAMES):
    y, u, gx, gv, grads = _run(dtype, kind, c, prm, saved_form, eps, want, use_u)
    p64 = {k: None if v is None else v[1] for k, v in prm.items()}
    x, v, gy, gu = (c[k][1] for k in ("x", "v", "gy", "gu"))
    yr, ur = ref.norm_residual(p64, kind, eps, x, v)
    # one fp32 rounding of v's deviation from its mean shows as 2^-24 |mean| / deviation
    rel = float(np.max(abs(v).max(1) / (np.std(v, axis=1) + eps ** 0.5))) if kind == "layer" else 1.0
    extra = 8 * 2.0 ** -24 * rel
    close("y", y, yr, dtype, extra=extra)
    if use_u:
        rely = float(np.max(abs(yr).max(1) / (np.std(yr, axis=1) + eps ** 0.5))) if kind == "layer" else 1.0
        extra += 8 * 2.0 ** -24 * rely
        close("u", u, ur, dtype, extra=extra)
    xb, vb = (ref.round_trip(t, LOW[dtype]) for t in (x, v)) if saved_form else (x, v)
    g = ref.norm_residual_backward(p64, kind, eps, xb, vb, gy, gu if use_u else None)
    rms = lambda t: np.sqrt(np.mean(t ** 2))  # noqa: E731
    for k, t in (("gx", gx), ("gv", gv)):
        close(k, t, g[k][0], dtype, size=np.maximum(g[k][1], rms(g[k][0])), extra=extra)
    for k, t in grads.items():
        close("g_" + k, t, g[k][0], dtype, size=g[k][1] + abs(g[k][0]), extra=extra)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm(dtype, kind, shape):
    B, C, P = shape
    if C == 1 and kind == "layer":
        pytest.skip("one channel has no deviation: see test_norm_of_constant_rows")
    c, prm = norm_case(dtype, B, C, P, seed=B * 7919 + C)
    _check(dtype, kind, c, prm, saved_form=False)
    _check(dtype, kind, c, prm, saved_form=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("P", [None, 90])
@pytest.mark.parametrize("absent", [("b_post", "b_pre"), ("gate",), ("scale", "w_post"), NORM_NAMES])
def test_norm_with_absent_parameters(dtype, P, absent):
    c, prm = norm_case(dtype, 3, 40, P, seed=11, absent=absent)
    _check(dtype, "layer", c, prm, saved_form=False)
    _check(dtype, "rms", c, prm, saved_form=True)


@pytest.mark.parametrize("P", [None, 90])
def test_norm_without_u(P):
    c, prm = norm_case("f16", 2, 24, P, seed=12)
    _check("f16", "layer", c, prm, saved_form=False, use_u=False)
    _check("f16", "rms", c, prm, saved_form=True, use_u=False)


@pytest.mark.parametrize("P", [None, 200])
def test_norm_with_a_large_mean(P):
    c, prm = norm_case("f32", 2, 96, P, seed=13, mean=1000.0)
    _check("f32", "layer", c, prm, saved_form=False)


@pytest.mark.parametrize("P", [None, 65])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_of_constant_rows(P, kind):
    """v zero (or, for the layer norm, equal over the channels): v^ is 0 and y = x + scale gate b_post."""
    c, prm = norm_case("f32", 2, 24, P, seed=14)
    v = torch.full_like(c["v"][0], 2.5 if kind == "layer" else 0.0)
    c["v"] = (v, v.double().numpy())
    y, u, gx, gv, grads = _run("f32", kind, c, prm, False)
    sg, b = prm["scale"][1] * prm["gate"][1], prm["b_post"][1]
    want = c["x"][1] + (sg * b if P is None else (sg * b)[..., None])
    close("y", y, want, "f32")
    assert torch.isfinite(gv).all() and float(grads["w_post"].abs().max()) == 0.0


@pytest.mark.parametrize("P", [None, 130])
def test_norm_poison_stays_in_its_row(P):
    c, prm = norm_case("f16", 2, 40, P, seed=15)
    v = c["v"][0].clone()
    v[(1, 3) if P is None else (1, 3, 100)] = float("nan")
    c["v"] = (v, v.double().numpy())
    y, u, gx, gv, _ = _run("f16", "layer", c, prm, False)
    bad = np.zeros(tuple(v.shape), bool)
    bad[(1,) if P is None else (1, slice(None), 100)] = True
    for t in (y, u, gx, gv):
        assert (np.isnan(f64(t)) == bad).all()


@pytest.mark.parametrize("P", [None, 77])
def test_norm_writes_only_what_is_wanted(P):
    c, prm = norm_case("bf16", 2, 20, P, seed=16)
    x, v, gy, gu = (dev(c[k][0]) for k in ("x", "v", "gy", "gu"))
    p = _params(prm)
    N = fno.NormParams("layer", 1e-5, **p)
    gx, gv = torch.empty_like(x), torch.empty_like(x)
    ws = fno.fno_norm_residual_workspace_empty(x)
    full = {k: torch.empty_like(t) for k, t in p.items()}
    fno.fno_norm_residual_backward(N, x, v, gy, gu, gx, gv, fno.NormGrads(**full), ws)
    one, gate = torch.empty_like(x), torch.empty_like(p["gate"])
    fno.fno_norm_residual_backward(N, x, v, gy, gu, one, None, None, None)
    assert torch.equal(one, gx)
    fno.fno_norm_residual_backward(N, x, v, gy, gu, None, one, fno.NormGrads(gate=gate), ws)
    assert torch.equal(one, gv) and torch.equal(gate, full["gate"])
    fno.fno_norm_residual_backward(N, x, v, gy, gu, None, None, fno.NormGrads(gate=gate.zero_()), ws)
    assert torch.equal(gate, full["gate"])


def test_norm_runs_on_the_given_stream_and_twice_alike():
    c, prm = norm_case("f16", 3, 64, 5000, seed=17)
    first = _run("f16", "layer", c, prm, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = _run("f16", "layer", c, prm, True)
    s.synchronize()
    for a, b in zip(first[:4], second[:4]):
        assert torch.equal(a, b)
    assert all(torch.equal(first[4][k], second[4][k]) for k in first[4])


# ------------------------------------------------------------- channel mix

def _mix_case(dtype, B, I, O, P, add, seed=0):
    rng = np.random.default_rng(seed)
    return dict(x=stored(rng, (B, I, P), dtype, spread=True), A=stored(rng, (O, I), dtype, I ** -0.5),
                bias=stored(rng, (O,), dtype, 0.3), add=stored(rng, (B, O, P), dtype, spread=True) if add else None,
                gy=stored(rng, (B, O, P), dtype, 0.5))


def _mix_run(c, act, want=("gx", "gA", "gbias", "gadd")):
    d = {k: None if t is None else dev(t[0]) for k, t in c.items()}
    O, add = d["A"].shape[0], d["add"] is not None
    y = torch.full_like(d["gy"], 7.0)
    saved = torch.full_like(fno.fno_channel_mix_saved_empty(d["x"], O, act, add), 99)
    fno.fno_channel_mix_save(d["x"], d["A"], d["bias"], d["add"], y, saved, act)
    out = {"gx": d["x"], "gA": d["A"], "gbias": d["bias"], "gadd": d["add"]}
    out = {k: torch.full_like(t, 7.0) if t is not None and k in want else None for k, t in out.items()}
    ws = torch.full_like(fno.fno_channel_mix_workspace_empty(d["x"], O), 255)
    fno.fno_channel_mix_backward_saved(saved, d["A"], d["bias"], d["gy"], out["gx"], out["gA"], out["gbias"], out["gadd"],
                                       ws, act, add)
    return y, out


# GELU and its derivative: fp32 to a few roundings; 16-bit types to 1e-6 (the
# published approximations' error in fp32), relative to |z| + 1
ACT = {"f32": 0.0, "f16": 1e-6, "bf16": 1e-6}


def _mix_check(dtype, B, I, O, P, act, add, seed=0):
    c = _mix_case(dtype, B, I, O, P, add, seed)
    y, out = _mix_run(c, act)
    v = {k: None if t is None else t[1] for k, t in c.items()}
    x, A, b, ad, gy = (v[k] for k in ("x", "A", "bias", "add", "gy"))
    a0 = 0.0 if ad is None else abs(ad)
    close("y", y, ref.channel_mix(x, A, b, ad, act), dtype, extra=ACT[dtype],
          size=ref.mix_pre(abs(x), abs(A), abs(b), None) + a0 + 1)
    xk = ref.round_trip(x, LOW[dtype])
    adk = ref.round_trip(ad, LOW[dtype]) if add and act else ad
    (gx, gA, gb, gz), _ = ref.channel_mix_backward(xk, A, b, adk, gy, act)
    # gz: slope's error times gy, z's own error (slope of slope below 1) times gy
    zs = ref.mix_pre(abs(xk), abs(A), abs(b), None) + a0 + 1
    gzs = abs(gy) * (zs if act else 1.0)
    close("gx", out["gx"], gx, dtype, extra=ACT[dtype], size=np.einsum("oi,bop->bip", abs(A), gzs))
    close("gA", out["gA"], gA, dtype, extra=ACT[dtype], size=np.einsum("bop,bip->oi", gzs, abs(xk)))
    close("gbias", out["gbias"], gb, dtype, extra=ACT[dtype], size=gzs.sum((0, 2)))
    if add:
        close("gadd", out["gadd"], gz, dtype, extra=ACT[dtype], size=gzs)


MIXES = [(2, 4, 4, 256), (1, 1, 1, 1), (1, 2, 3, 31), (3, 5, 7, 33), (2, 16, 16, 64), (1, 17, 16, 65), (2, 16, 17, 300),
         (1, 32, 32, 1024), (2, 33, 31, 127), (5, 40, 72, 201), (1, 64, 64, 129), (1, 65, 64, 100), (1, 64, 65, 100),
         (1, 128, 128, 70), (2, 128, 3, 90), (2, 3, 128, 90), (1, 128, 20, 333), (1, 20, 100, 257), (9, 8, 48, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act,add", [(1, True), (1, False), (0, True), (0, False)])
@pytest.mark.parametrize("shape", MIXES, ids=str)
def test_mix(dtype, shape, act, add):
    _mix_check(dtype, *shape, act, add, seed=sum(shape))


@pytest.mark.parametrize("dtype", DTYPES)
def test_mix_over_many_tiles(dtype):
    _mix_check(dtype, 3, 24, 40, 20011, 1, True, seed=5)


@pytest.mark.parametrize("want", [("gx",), ("gA",), ("gbias",), ("gadd",), ("gx", "gadd"), ("gA", "gbias")])
def test_mix_writes_only_what_is_wanted(want):
    c = _mix_case("f16", 2, 24, 40, 150, True, seed=6)
    _, full = _mix_run(c, 1)
    _, some = _mix_run(c, 1, want)
    for k in full:
        assert some[k] is None if k not in want else torch.equal(some[k], full[k]), k


@pytest.mark.parametrize("dtype", DTYPES)
def test_mix_without_bias(dtype):
    c = _mix_case(dtype, 2, 12, 20, 70, True, seed=7)
    zero = torch.zeros_like(c["bias"][0])
    with_zero = _mix_run({**c, "bias": (zero, None)}, 1)
    none = _mix_run({**c, "bias": None}, 1)
    assert torch.equal(with_zero[0], none[0])
    assert all(torch.equal(with_zero[1][k], none[1][k]) for k in ("gx", "gA", "gadd"))


def test_mix_large_and_saturated_z():
    """Far out GELU is the identity or zero and its slope one or zero; nothing overflows on the way."""
    c = _mix_case("f32", 1, 4, 4, 64, True, seed=8)
    a = c["add"][0].clone()
    a[0, :, :16], a[0, :, 16:32], a[0, :, 32:48], a[0, :, 48:] = 1e4, -1e4, 1e30, -1e30
    c["add"] = (a, a.double().numpy())
    y, out = _mix_run(c, 1)
    gy = c["gy"][0].to(DEV)
    up = (a > 0).to(DEV)
    assert torch.isfinite(y).all() and (y[~up] == 0).all()
    assert torch.equal(out["gadd"][up], gy[up]) and (out["gadd"][~up] == 0).all()


def test_mix_poison():
    """A NaN in x poisons its block of that channel, so z, and with it every gradient
    through those pixels; other pixels stay what they are."""
    c = _mix_case("f16", 1, 5, 6, 100, True, seed=9)
    clean = _mix_run(c, 1)
    x = c["x"][0].clone()
    x[0, 2, 40] = float("nan")
    y, out = _mix_run({**c, "x": (x, None)}, 1)
    assert torch.isnan(y[0, :, 40]).all() and torch.equal(y[0, :, 41:], clean[0][0, :, 41:])
    hit = torch.zeros(100, dtype=torch.bool, device=DEV)
    hit[32:64] = True
    for k in ("gx", "gadd"):
        assert torch.isnan(out[k][0][:, hit]).all() and torch.equal(out[k][0][:, ~hit], clean[1][k][0][:, ~hit])


def test_mix_twice_alike():
    c = _mix_case("bf16", 4, 48, 64, 3000, True, seed=10)
    (ya, a), (yb, b) = _mix_run(c, 1), _mix_run(c, 1)
    assert torch.equal(ya, yb) and all(torch.equal(a[k], b[k]) for k in a)


def test_mix_gradients_against_differences():
    """The whole operator in fp32 against a central difference of its own forward, at values
    that a checkpoint keeps exactly."""
    c = _mix_case("f32", 2, 6, 5, 50, True, seed=11)
    for k in ("x", "add"):
        kept = torch.from_numpy(ref.round_trip(c[k][1], -126)).float()
        c[k] = (kept, kept.double().numpy())
    y, out = _mix_run(c, 1)
    rng = np.random.default_rng(12)
    h = 1e-4
    for name, key in (("A", "gA"), ("bias", "gbias"), ("x", "gx"), ("add", "gadd")):
        d = rng.standard_normal(c[name][1].shape)
        loss = [(ref.channel_mix(*(c[k][1] + (s * h * d if k == name else 0) for k in ("x", "A", "bias", "add")), 1)
                 * c["gy"][1]).sum() for s in (-1, 1)]
        diff = (loss[1] - loss[0]) / (2 * h)
        got = (f64(out[key]) * d).sum()
        # h^2 of the third derivative, and fp32 sums
        assert abs(got - diff) <= 1e-5 * (abs(f64(out[key]) * d)).sum()


@pytest.mark.parametrize("scale_x,scale_gy", [(2.0 ** -18, 1.0), (1.0, 2.0 ** -12), (2.0 ** 7, 2.0 ** 14)])
def test_mix_at_the_ends_of_fp16(scale_x, scale_gy):
    """Subnormal inputs are used as they are; gz near the type's largest does not overflow on its way to gA
    and gx (weights and x small enough that those are finite)."""
    c = _mix_case("f16", 1, 20, 24, 100, True, seed=13)
    for k, s in (("x", scale_x), ("add", min(scale_x, 1.0)), ("gy", scale_gy)):
        t = (c[k][0].double().clamp(-3.9, 3.9) * s).half()
        c[k] = (t, t.double().numpy())
    small = (c["A"][0].double() / 64).half()
    c["A"] = (small, small.double().numpy())
    if scale_x > 1:
        tiny = (c["x"][0].double() * 2.0 ** -20).half()
        c["x"] = (tiny, tiny.double().numpy())
    y, out = _mix_run(c, 1)
    v = {k: t[1] for k, t in c.items()}
    xk, adk = ref.round_trip(v["x"], -24), ref.round_trip(v["add"], -24)
    (gx, gA, gb, gz), _ = ref.channel_mix_backward(xk, v["A"], v["bias"], adk, v["gy"], 1)
    zs = ref.mix_pre(abs(xk), abs(v["A"]), abs(v["bias"]), None) + abs(v["add"]) + 1
    gzs = abs(v["gy"]) * zs
    # fp16's largest, 65504, bounds the outputs that can be compared
    assert max(abs(gx).max(), abs(gA).max()) < 65504
    close("gx", out["gx"], gx, "f16", extra=ACT["f16"], size=np.einsum("oi,bop->bip", abs(v["A"]), gzs))
    close("gA", out["gA"], gA, "f16", extra=ACT["f16"], size=np.einsum("bop,bip->oi", gzs, abs(xk)))


@pytest.mark.parametrize("dtype", DTYPES)
def test_mix_of_infinities(dtype):
    """GELU of plus infinity is infinite, of minus infinity its limit, 0; the block that held
    one reads back as NaN, so the gradients through its pixels are NaN and others are as before."""
    c = _mix_case(dtype, 1, 5, 6, 100, True, seed=14)
    clean = _mix_run(c, 1)
    a = c["add"][0].clone()
    a[0, 1, 40], a[0, 2, 41] = float("inf"), -float("inf")
    y, out = _mix_run({**c, "add": (a, None)}, 1)
    assert y[0, 1, 40] == float("inf") and y[0, 2, 41] == 0
    same = torch.ones_like(y, dtype=torch.bool)
    same[0, 1, 40] = same[0, 2, 41] = False
    assert torch.equal(y[same], clean[0][same])
    hit = torch.zeros(100, dtype=torch.bool, device=DEV)
    hit[32:64] = True
    assert torch.isnan(out["gadd"][0, 1:3, hit]).all() and torch.equal(out["gx"][0][:, ~hit], clean[1]["gx"][0][:, ~hit])
    assert torch.equal(out["gadd"][0, 3:], clean[1]["gadd"][0, 3:])
