"""The definitions of oracle/training.py on torch float64 tensors, for cases of millions of
values (tests/test_training_ref64_cpu.py holds them against the oracle), and the shapes that
reach every kernel of the training operators."""

import math

import torch

from training_util import CHAIN, NORM_NAMES, half_step

# ------------------------------------------------------------- definitions


def round_trip(x, low):
    n = x.shape[-1]
    b = torch.nn.functional.pad(x, (0, -n % 32)).unflatten(-1, (-1, 32))
    big = b.abs().amax(-1, keepdim=True)
    e = torch.where(big > 0, torch.frexp(big).exponent - 7, low).clamp(min=low).double()  # floor(log2 big) - 6
    step = torch.exp2(e)
    return ((b / step).round().clamp(-127, 127) * step).flatten(-2)[..., :n]


def _unit(h, kind, eps):
    m = h.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(h[:, :1])
    r = 1 / (((h - m) ** 2).mean(1, keepdim=True) + eps).sqrt()
    return (h - m) * r, r


def _wide(p, ndim, none):
    if p is None:
        return none
    p = p if p.dim() == 2 else p[None]
    return p[..., None] if ndim == 3 else p


def norm_residual(prm, kind, eps, x, v):
    at = lambda k, none: _wide(prm.get(k), x.dim(), none)  # noqa: E731
    vh, _ = _unit(v, kind, eps)
    y = x + at("scale", 1.0) * at("gate", 1.0) * (vh * at("w_post", 1.0) + at("b_post", 0.0))
    return y, _unit(y, kind, eps)[0] * at("w_pre", 1.0) + at("b_pre", 0.0)


def norm_residual_backward(prm, kind, eps, x, v, gy, gu):
    """{name: (gradient, size of the terms it is summed from)}."""
    at = lambda k, none: _wide(prm.get(k), x.dim(), none)  # noqa: E731
    layer = kind == "layer"

    def through(g, h, r, size=False):
        t = g.abs() + h.abs() * (g * h).abs().mean(1, keepdim=True) if size else g - h * (g * h).mean(1, keepdim=True)
        if layer:
            t = t + g.abs().mean(1, keepdim=True) if size else t - g.mean(1, keepdim=True)
        return r * t

    mag = lambda t: t.abs() if torch.is_tensor(t) else abs(t)  # noqa: E731
    vh, r = _unit(v, kind, eps)
    sg = at("scale", 1.0) * at("gate", 1.0)
    n = vh * at("w_post", 1.0) + at("b_post", 0.0)
    vh_size = r * (v.abs() + (v.mean(1, keepdim=True).abs() if layer else 0.0))
    n_size = vh_size * mag(at("w_post", 1.0)) + mag(at("b_post", 0.0))
    col, per = ((0, 2), (2,)) if x.dim() == 3 else ((0,), ())
    both = lambda t, s, axes: (t.sum(axes), s.sum(axes)) if axes else (t, s)  # noqa: E731
    out, gx, gx_size = {}, gy, gy.abs()
    if gu is not None:
        yh, ry = _unit(x + sg * n, kind, eps)
        g = gu * at("w_pre", 1.0)
        yh_size = ry * (x.abs() + mag(sg) * n_size) * (2.0 if layer else 1.0)
        gx, gx_size = gy + through(g, yh, ry), gy.abs() + through(g, yh_size, ry, True)
        out["w_pre"], out["b_pre"] = both(gu * yh, gu.abs() * yh_size, col), both(gu, gu.abs(), col)
    gn, gn_size = gx * sg, gx_size * mag(sg)
    h, h_size = gn * at("w_post", 1.0), gn_size * mag(at("w_post", 1.0))
    out.update(gx=(gx, gx_size), gv=(through(h, vh, r), through(h_size, vh_size, r, True)),
               w_post=both(gn * vh, gn_size * vh_size, col), b_post=both(gn, gn_size, col),
               gate=both(gx * at("scale", 1.0) * n, gx_size * mag(at("scale", 1.0)) * n_size, per),
               scale=both(gx * at("gate", 1.0) * n, gx_size * mag(at("gate", 1.0)) * n_size, col))
    return out


def mix_pre(x, A, bias, add):
    z = torch.matmul(A, x)
    z = z if bias is None else z + bias[:, None]
    return z if add is None else z + add


def channel_mix(x, A, bias, add, act):
    z = mix_pre(x, A, bias, add)
    return z * torch.special.ndtr(z) if act else z


def channel_mix_backward(x, A, bias, add, gy, act):
    """gx, gA, gbias, gz."""
    gz = gy
    if act:
        z = mix_pre(x, A, bias, add)
        gz = gy * (torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
    return (torch.matmul(A.t().contiguous(), gz), torch.einsum("bop,bip->oi", gz, x), gz.sum((0, 2)), gz)


def close(name, got, ref, dtype, size=None, extra=0.0):
    """training_util.close() on float64 tensors."""
    got = got.double()
    assert got.shape == ref.shape, name
    if size is None:
        size = torch.maximum(ref.abs(), ref.square().mean().sqrt())
    step = 2.0 ** -25 if dtype == "f16" else 0.0
    off = (got - ref).abs() - (half_step(dtype) * ref.abs() * (1 + 2.0 ** -10) + (CHAIN + extra) * size + step)
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    assert bool((off <= 0).all()), (f"{name}: off by {float((got - ref).abs().max()):.3g}, {int((off > 0).sum())} of "
                                    f"{off.numel()} over the bound by up to {float(off.max()):.3g}")


def check_norm(run, dtype, kind, c, prm, low, eps=1e-5, saved_form=False):
    """run's (y, u, gx, gv, grads) against the definitions; c and prm hold (tensor, float64) pairs. Bounds as in
    test_gpu_training: one fp32 rounding of a deviation from the mean shows as 2^-24 |mean| / deviation."""
    y, u, gx, gv, grads = run
    p64 = {k: None if t is None else t[1] for k, t in prm.items()}
    x, v, gy, gu = (c[k][1] for k in ("x", "v", "gy", "gu"))
    yr, ur = norm_residual(p64, kind, eps, x, v)
    rel = lambda t: float((t.abs().amax(1) / (t.std(1, correction=0) + eps ** 0.5)).max()) if kind == "layer" else 1.0  # noqa: E731
    extra = 8 * 2.0 ** -24 * rel(v)
    close("y", y, yr, dtype, extra=extra)
    extra += 8 * 2.0 ** -24 * rel(yr)
    close("u", u, ur, dtype, extra=extra)
    if saved_form:
        x, v = round_trip(x, low), round_trip(v, low)
    g = norm_residual_backward(p64, kind, eps, x, v, gy, gu)
    for k, t in (("gx", gx), ("gv", gv)):
        close(k, t, g[k][0], dtype, size=torch.maximum(g[k][1], g[k][0].square().mean().sqrt()), extra=extra)
    for k, t in grads.items():
        close("g_" + k, t, g[k][0], dtype, size=g[k][1] + g[k][0].abs(), extra=extra)


def check_norm_small(run, dtype, kind, c, prm, low, eps=1e-5, saved_form=False):
    """check_norm() with errors followed to first order, for few channels, where y or a deviation from the mean may
    vanish in all of them (a pixel in a million) and a norm then magnifies what rounding left. U = 2^-24; a sum over C <= 8
    channels is off by at most 8 U of its terms' sizes, products of parameters by U for each factor; sums over
    samples and pixels by CHAIN of theirs. E_q is the error of q, rho that of an inverse deviation r relative to it."""
    U, layer = 2.0 ** -24, kind == "layer"
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    p = {k: t[1] for k, t in prm.items()}
    at = lambda k: _wide(p[k], c["x"][1].dim(), None)  # noqa: E731
    w, b, sg, wp, bp = at("w_post"), at("b_post"), at("scale") * at("gate"), at("w_pre"), at("b_pre")

    def unit(h, E_h):  # h^, r, E of h^, rho
        hh, r = _unit(h, kind, eps)
        E_d = E_h + U * hh.abs() / r + (mean(E_h) + 8 * U * mean(h.abs()) if layer else 0.0)
        rho = r * mean(hh.abs() * E_d) + 8 * U
        return hh, r, r * E_d + hh.abs() * (rho + 2 * U), rho

    def forward(x, v):
        vh, r, E_vh, rho = unit(v, torch.zeros_like(v))
        n, n_size = vh * w + b, (vh * w).abs() + b.abs()
        E_n = w.abs() * E_vh + 3 * U * n_size
        y = x + sg * n
        E_y = sg.abs() * (w.abs() * E_vh + 6 * U * n_size) + U * (x.abs() + y.abs())
        return (vh, r, E_vh, rho), (n, E_n), (y, E_y), unit(y, E_y)

    def through(g, E_g, hh, r, E_hh, rho):
        m1 = mean(g * hh)
        E_m1 = mean(hh.abs() * E_g + g.abs() * E_hh) + 8 * U * mean((g * hh).abs())
        t, size = g - hh * m1, g.abs() + (hh * m1).abs()
        E_t = E_g + hh.abs() * E_m1 + m1.abs() * E_hh
        if layer:
            t, size, E_t = t - mean(g), size + mean(g).abs(), E_t + mean(E_g) + 8 * U * mean(g.abs())
        return r * t, r * (E_t + 3 * U * size) + (r * t).abs() * (rho + 2 * U)

    def held(name, got, ref, E):
        got, ref = got.double(), ref.reshape(got.shape)
        bound = half_step(dtype) * ref.abs() * (1 + 2.0 ** -10) + 1.0625 * E.reshape(got.shape) + (2.0 ** -25 if dtype == "f16" else 0.0)
        off = (got - ref).abs() / bound
        assert bool(torch.isfinite(got).all()), f"{name}: not finite"
        assert bool((off <= 1).all()), f"{name}: {int((off > 1).sum())} of {off.numel()} over the bound, by {float(off.max()):.3g}"

    y_, u_, gx_, gv_, grads = run
    x, v, gy, gu = (c[k][1] for k in ("x", "v", "gy", "gu"))
    _, _, (y, E_y), (yh, ry, E_yh, rho_y) = forward(x, v)
    held("y", y_, y, E_y)
    held("u", u_, yh * wp + bp, wp.abs() * E_yh + 2 * U * ((wp * yh).abs() + bp.abs()))
    if saved_form:
        (vh, r, E_vh, rho), (n, E_n), _, (yh, ry, E_yh, rho_y) = forward(round_trip(x, low), round_trip(v, low))
    else:
        (vh, r, E_vh, rho), (n, E_n), _, _ = forward(x, v)
    g = gu * wp
    t, E_t = through(g, U * g.abs(), yh, ry, E_yh, rho_y)
    gx, E_gx = gy + t, E_t + U * (gy + t).abs()
    h = gx * sg * w
    E_h = (sg * w).abs() * E_gx + 4 * U * h.abs()
    held("gx", gx_, gx, E_gx)
    held("gv", gv_, *through(h, E_h, vh, r, E_vh, rho))
    col, per = ((0, 2), (2,)) if x.dim() == 3 else ((0,), ())
    n_size = (vh * w).abs() + b.abs()
    gate, scale = at("gate"), at("scale")
    for k, f, term, E, size, axes in (
            ("gate", scale, gx * n, E_gx * n.abs() + gx.abs() * E_n, gx.abs() * n_size, per),
            ("scale", gate, gx * n, E_gx * n.abs() + gx.abs() * E_n, gx.abs() * n_size, col),
            ("w_post", sg, gx * vh, E_gx * vh.abs() + gx.abs() * E_vh, (gx * vh).abs(), col),
            ("b_post", sg, gx, E_gx, gx.abs(), col), ("w_pre", 1.0, gu * yh, gu.abs() * E_yh, (gu * yh).abs(), col),
            ("b_pre", 1.0, gu, torch.zeros_like(gu), gu.abs(), col)):
        ref, err = f * term, abs(f) * (E + CHAIN * size)
        held("g_" + k, grads[k], ref.sum(axes) if axes else ref, err.sum(axes) if axes else err)


# ------------------------------------------------------------------- shapes

# Fields. A tile is 32 (fp32) or 64 pixels; a wave of a workgroup has W C / 8 of its channels. Up to
# 64 channels have one wave a tile (four tiles a workgroup), 128 two, 256 four and 512 eight, but
# 9 to 128 channels with fewer than 512 tiles in all four.
#   FEW: fewer than 512 tiles;  MANY: more, and with 2052 samples one workgroup a sample, so that
# each wave goes over two or more tiles, the last of them ragged.
SMALL_CHANNELS = (1, 2, 3, 5, 8)  # one group of eight: checked with the bounds of check_norm_small()
FEW_CHANNELS = (9, 30, 62, 95, 128)
MANY_CHANNELS = (14, 17, 32, 33, 48, 55, 61, 66, 90, 112, 125, 130, 170, 219, 256, 257, 380, 420, 509)


def field_tile(dtype):
    return 32 if dtype == "f32" else 64


def few(C, dtype):
    return 2, C, 5 * field_tile(dtype) + 7


def many(C, dtype):
    return 2052, C, (4 if C <= 64 else 1) * field_tile(dtype) + 9


# one sample's row over all 4096 workgroups, and more than one round of tiles in each
def long_row(C, dtype):
    return 1, C, 4096 * 4 * field_tile(dtype) + 77


# Tokens: (channels, rows); the rows give each workgroup of the forward, and so of the backward, a second row.
TOKENS = {"f32": ((5, 17000), (255, 17000), (510, 8500), (1022, 4300), (2047, 2200), (4093, 1100), (8190, 2200)),
          "f16": ((5, 17000), (510, 17000), (1022, 8500), (2047, 4300), (4093, 2200), (8190, 1100))}
TOKENS["bf16"] = TOKENS["f16"]

# Channel mix: channels on either side, in tiles of 16 (1, 2, 4 or 8 of them)
MIX_CHANNELS = (13, 30, 52, 120)


def mix_many(O, dtype):
    """(batch, pixels) of more than 4096 tiles of the forward, whole and ragged in turn."""
    wide = O <= 16 and 256 or O <= 32 and 128 or O <= 64 and (128 if dtype != "f32" else 64) or 64
    return 2100, wide + 5
