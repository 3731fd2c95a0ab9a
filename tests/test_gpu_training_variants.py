"""Every kernel of the training operators against float64, at shapes that give a workgroup
several tiles or rows (tests/test_training_variants_cpu.py shows which kernels these are):
sums carried from tile to tile, double buffers, loads a tile ahead, ragged last tiles and channels."""

import pytest
import torch

import training_ref64 as r64
from test_gpu_training import _mix_run, _run
from training_util import DT, LOW, NORM_NAMES

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]


def _stored(gen, shape, dtype, scale=1.0, mean=0.0, spread=False):
    t = torch.randn(shape, generator=gen, device="cuda") * scale + mean
    if spread:
        t *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    t = t.to(DT[dtype])
    return t, t.double()


def _norm(dtype, kind, B, C, P, saved_form, check=r64.check_norm):
    gen = torch.Generator(device="cuda").manual_seed(B * 31 + C)
    shape = (B, C) if P is None else (B, C, P)
    c = {k: _stored(gen, shape, dtype, s) for k, s in (("x", 1.0), ("v", 3.0), ("gy", 0.5), ("gu", 0.5))}
    prm = {k: _stored(gen, s, dtype, dev, mid) for k, mid, dev, s in
           (("w_post", 1.0, 0.2, (C,)), ("b_post", 0.0, 0.1, (C,)), ("gate", 0.5, 0.3, (B, C)), ("scale", 0.2, 0.05, (C,)),
            ("w_pre", 1.0, 0.2, (C,)), ("b_pre", 0.0, 0.1, (C,)))}
    assert set(prm) == set(NORM_NAMES)
    check(_run(dtype, kind, c, prm, saved_form), dtype, kind, c, prm, LOW[dtype], saved_form=saved_form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("C", r64.FEW_CHANNELS)
def test_norm_on_few_tiles(dtype, kind, C):
    for saved_form in (False, True):
        _norm(dtype, kind, *r64.few(C, dtype), saved_form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind,C", [(k, C) for k in ("rms", "layer") for C in r64.SMALL_CHANNELS if k == "rms" or C > 1])
def test_norm_on_many_tiles_of_few_channels(dtype, kind, C):
    for saved_form in (False, True):
        _norm(dtype, kind, *r64.many(C, dtype), saved_form, r64.check_norm_small)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("C", r64.MANY_CHANNELS)
def test_norm_on_many_tiles(dtype, kind, C):
    for saved_form in (False, True):
        _norm(dtype, kind, *r64.many(C, dtype), saved_form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_on_one_long_field(dtype, kind):
    _norm(dtype, kind, *r64.long_row(10, dtype), kind == "rms")


@pytest.mark.parametrize("dtype,C,rows", [(d, *s) for d in DTYPES for s in r64.TOKENS[d]])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_on_many_tokens(dtype, kind, C, rows):
    for saved_form in (False, True):
        _norm(dtype, kind, rows, C, None, saved_form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("O", r64.MIX_CHANNELS)
@pytest.mark.parametrize("I", r64.MIX_CHANNELS)
@pytest.mark.parametrize("act,add", [(1, True), (0, True), (1, False)])
def test_mix_on_many_tiles(dtype, O, I, act, add):
    B, P = r64.mix_many(O, dtype)
    gen = torch.Generator(device="cuda").manual_seed(O * 131 + I)
    c = dict(x=_stored(gen, (B, I, P), dtype, spread=True), A=_stored(gen, (O, I), dtype, I ** -0.5),
             bias=_stored(gen, (O,), dtype, 0.3), add=_stored(gen, (B, O, P), dtype, spread=True) if add else None,
             gy=_stored(gen, (B, O, P), dtype, 0.5))
    y, out = _mix_run(c, act)
    x, A, b, ad, gy = (None if c[k] is None else c[k][1] for k in ("x", "A", "bias", "add", "gy"))
    a0 = 0.0 if ad is None else ad.abs()
    # bounds as in test_gpu_training; GELU and its derivative to a few roundings in every type
    r64.close("y", y, r64.channel_mix(x, A, b, ad, act), dtype, size=r64.mix_pre(x.abs(), A.abs(), b.abs(), None) + a0 + 1)
    xk = r64.round_trip(x, LOW[dtype])
    adk = r64.round_trip(ad, LOW[dtype]) if add and act else ad
    gx, gA, gb, gz = r64.channel_mix_backward(xk, A, b, adk, gy, act)
    gzs = gy.abs() * (r64.mix_pre(xk.abs(), A.abs(), b.abs(), None) + a0 + 1 if act else 1.0)
    r64.close("gx", out["gx"], gx, dtype, size=torch.matmul(A.abs().t().contiguous(), gzs))
    r64.close("gA", out["gA"], gA, dtype, size=torch.einsum("bop,bip->oi", gzs, xk.abs()))
    r64.close("gbias", out["gbias"], gb, dtype, size=gzs.sum((0, 2)))
    if add:
        r64.close("gadd", out["gadd"], gz, dtype, size=gzs)
