"""float64 definitions of the training operators around a block: the 8-bit
checkpoint format, the channel mix with GELU and its gradients, and the norms
with gate and residual scale and theirs. Written from the formulas, with the
sizes of the sums' terms (for error bounds) where a result is a long sum."""

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ------------------------------------------------------------- checkpoints

def checkpoint(x, low):
    """(codes, exponents) of x [rows][n] float64; codes [rows][32 nb]."""
    rows, n = x.shape
    nb = -(-n // 32)
    b = np.zeros((rows, nb * 32))
    b[:, :n] = x
    b = b.reshape(rows, nb, 32)
    e = np.empty((rows, nb), np.int64)
    q = np.empty(b.shape, np.int64)
    for r in range(rows):
        for k in range(nb):
            big = np.max(np.abs(b[r, k]))
            if not np.isfinite(big):
                e[r, k], q[r, k] = 127, 0
                continue
            e[r, k] = low if big == 0 else max(math.floor(math.log2(big)) - 6, low)
            if big != 0 and 2.0 ** (e[r, k] + 7) <= big:  # log2 rounded down past a power of two
                e[r, k] += 1
            q[r, k] = np.clip(np.rint(b[r, k] * 2.0 ** -float(e[r, k])), -127, 127)
    return q.reshape(rows, nb * 32), e


def checkpoint_values(codes, exps, n):
    rows, nb = exps.shape
    step = np.where(exps == 127, np.nan, 2.0 ** exps.astype(np.float64))
    return (codes.reshape(rows, nb, 32) * step[..., None]).reshape(rows, nb * 32)[:, :n]


def round_trip(x, low):
    """The values a checkpoint of x [..., n] keeps."""
    flat = x.reshape(-1, x.shape[-1])
    return checkpoint_values(*checkpoint(flat, low), flat.shape[1]).reshape(x.shape)


# ------------------------------------------------------------- channel mix

def gelu_slope(z):
    return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def mix_pre(x, A, bias, add):
    """z [B][Co][P] = A x + bias + add."""
    z = np.einsum("oi,bip->bop", A, x)
    if bias is not None:
        z = z + bias[None, :, None]
    return z if add is None else z + add


def channel_mix(x, A, bias, add, act):
    z = mix_pre(x, A, bias, add)
    return 0.5 * z * (1 + _erf(z / math.sqrt(2))) if act else z


def channel_mix_backward(x, A, bias, add, gy, act):
    """(gx, gA, gbias, gadd) and the sums of the terms' sizes of gx, gA, gbias."""
    gz = gy * gelu_slope(mix_pre(x, A, bias, add)) if act else gy
    sums = (np.einsum("oi,bop->bip", A, gz), np.einsum("bop,bip->oi", gz, x), gz.sum((0, 2)))
    size = (np.einsum("oi,bop->bip", abs(A), abs(gz)), np.einsum("bop,bip->oi", abs(gz), abs(x)),
            abs(gz).sum((0, 2)))
    return sums + (gz,), size


# -------------------------------------------------------------------- norms

def _unit(h, kind, eps):
    m = h.mean(1, keepdims=True) if kind == "layer" else 0.0
    r = 1 / np.sqrt(((h - m) ** 2).mean(1, keepdims=True) + eps)
    return (h - m) * r, r


def _wide(p, ndim, none):
    if p is None:
        return none
    p = p if p.ndim == 2 else p[None]
    return p[..., None] if ndim == 3 else p


def norm_residual(prm, kind, eps, x, v):
    """(y, u); prm: dict with w_post, b_post, gate, scale, w_pre, b_pre (None where absent)."""
    at = lambda k, none: _wide(prm.get(k), x.ndim, none)  # noqa: E731
    vh, _ = _unit(v, kind, eps)
    y = x + at("scale", 1.0) * at("gate", 1.0) * (vh * at("w_post", 1.0) + at("b_post", 0.0))
    yh, _ = _unit(y, kind, eps)
    return y, yh * at("w_pre", 1.0) + at("b_pre", 0.0)


def _through(g, h, r, kind):
    t = g - h * (g * h).mean(1, keepdims=True)
    return r * (t - g.mean(1, keepdims=True) if kind == "layer" else t)


def _terms(g, h, r, kind):
    """Size of the terms _through adds up (they cancel where few channels share a norm)."""
    t = abs(g) + abs(h) * (abs(g * h)).mean(1, keepdims=True)
    return r * (t + abs(g).mean(1, keepdims=True) if kind == "layer" else t)


def norm_residual_backward(prm, kind, eps, x, v, gy, gu):
    """Gradients gx, gv and those of the parameters, each as (value, size of the terms it is summed from)."""
    at = lambda k, none: _wide(prm.get(k), x.ndim, none)  # noqa: E731
    vh, r = _unit(v, kind, eps)
    n = vh * at("w_post", 1.0) + at("b_post", 0.0)
    sg = at("scale", 1.0) * at("gate", 1.0)
    gx, gx_size = gy, abs(gy)
    out = {}
    col, per = ((0, 2), (2,)) if x.ndim == 3 else ((0,), ())
    vh_size = r * (abs(v) + (abs(v.mean(1, keepdims=True)) if kind == "layer" else 0.0))
    n_size = vh_size * abs(at("w_post", 1.0)) + abs(at("b_post", 0.0))
    both = lambda t, size, axes: (t.sum(axes), size.sum(axes)) if axes else (t, size)  # noqa: E731
    if gu is not None:
        yh, ry = _unit(x + sg * n, kind, eps)
        g = gu * at("w_pre", 1.0)
        yh_size = ry * (abs(x) + abs(sg) * n_size) * (2.0 if kind == "layer" else 1.0)
        gx, gx_size = gy + _through(g, yh, ry, kind), abs(gy) + _terms(g, yh_size, ry, kind)
        out["w_pre"], out["b_pre"] = both(gu * yh, abs(gu) * yh_size, col), both(gu, abs(gu), col)
    gn, gn_size = gx * sg, gx_size * abs(sg)
    h, h_size = gn * at("w_post", 1.0), gn_size * abs(at("w_post", 1.0))
    out.update(gx=(gx, gx_size), gv=(_through(h, vh, r, kind), _terms(h_size, vh_size, r, kind)),
               w_post=both(gn * vh, gn_size * vh_size, col), b_post=both(gn, gn_size, col),
               gate=both(gx * at("scale", 1.0) * n, gx_size * abs(at("scale", 1.0)) * n_size, per),
               scale=both(gx * at("gate", 1.0) * n, gx_size * abs(at("gate", 1.0)) * n_size, col))
    return out
