"""float64 definitions of the operators of a regularised block and of its 4-bit serving
form: counter-based dropout, group norm with an activation and its gradients, and
microscaled 4-bit floats. Written from the formulas, with the sizes of the terms (for error
bounds) beside the results."""

import math

import numpy as np

from .training import gelu_slope

_erf = np.vectorize(math.erf, otypes=[np.float64])
_LOW = np.uint64(0xFFFFFFFF)


# ------------------------------------------------------------------- dropout

def philox(block, offset, seed):
    """Philox 4x32-10 (Salmon, Moraes, Dror, Shaw, SC 2011): the four 32-bit words [..., 4] at counter
    (block, offset) and key seed, 64 bits each, low words first."""
    block = np.asarray(block, np.uint64)
    split = lambda v: (np.full(block.shape, v & 0xFFFFFFFF, np.uint64), np.full(block.shape, v >> 32, np.uint64))  # noqa: E731
    c = [block & _LOW, block >> np.uint64(32), *split(offset)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        p0, p2 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)  # below 2^64
        c = [(p2 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p2 & _LOW,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & _LOW]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, -1)


def drop_threshold(p):
    return int(np.rint(float(np.float32(p)) * 65536))


def kept_units(n, p, seed, offset):
    """Which of units 0 .. n - 1 are kept."""
    w = philox(np.arange(-(-n // 8), dtype=np.uint64), offset, seed)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(-1)
    return bits[:n] >= drop_threshold(p)


def drop_factor(B, C, P, last, p, seed, offset=0, unit="element"):
    """D(v) = factor v, against [B][C][P] or [B][P][C] (last)."""
    t = drop_threshold(p)
    shape = {"element": (B, P, C) if last else (B, C, P), "channel": (B, 1, C) if last else (B, C, 1),
             "sample": (B, 1, 1)}[unit]
    if t == 0:
        return np.ones((1, 1, 1))
    scale = 65536 / (65536 - t) if t < 65536 else 0.0
    return np.where(kept_units(math.prod(shape), p, seed, offset).reshape(shape), scale, 0.0)


# ---------------------------------------------------------------- group norm

def act(z, kind):
    if kind == 1:
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    return z / (1 + np.exp(-z)) if kind == 2 else z


def act_slope(z, kind):
    if kind == 1:
        return gelu_slope(z)
    if kind == 2:
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def _grouped(t, groups, last):
    B = t.shape[0]
    if last:
        return t.reshape(B, t.shape[1], groups, -1), (1, 3)
    return t.reshape(B, groups, -1, t.shape[2]), (2, 3)


def group_norm(x, groups, eps, w, b, kind, last, factor=1.0):
    """(y, mean [B][G], r [B][G], size of y's terms) of x [B][C][P] or [B][P][C]."""
    B, C = x.shape[0], x.shape[2 if last else 1]
    g, axes = _grouped(x, groups, last)
    mean = g.mean(axes, keepdims=True)
    r = 1 / np.sqrt(((g - mean) ** 2).mean(axes, keepdims=True) + eps)
    h = ((g - mean) * r).reshape(x.shape)
    z, size = _affine(h, ((abs(g) + abs(mean)) * r).reshape(x.shape), w, b, last)
    return act(z, kind) * factor, mean.reshape(B, groups), r.reshape(B, groups), size * factor


def _affine(h, hs, w, b, last):
    at = (lambda p: p[None, None, :]) if last else (lambda p: p[None, :, None])
    w = 1.0 if w is None else at(w)
    b = 0.0 if b is None else at(b)
    return h * w + b, hs * abs(w) + abs(b)


def group_norm_backward(x, groups, eps, w, b, kind, last, gy, factor=1.0):
    """((gx, gw, gb), the sizes of their terms)."""
    g, axes = _grouped(x, groups, last)
    n = g.shape[axes[0]] * g.shape[axes[1]]
    mean = g.mean(axes, keepdims=True)
    r = 1 / np.sqrt(((g - mean) ** 2).mean(axes, keepdims=True) + eps)
    h, hs = (g - mean) * r, (abs(g) + abs(mean)) * r
    z, zs = _affine(h.reshape(x.shape), hs.reshape(x.shape), w, b, last)
    gy = gy * factor
    gz = gy * act_slope(z, kind)
    gzs = abs(gz) + (abs(gy) * zs if kind else 0.0)   # an error of z moves the slope
    over = (0, 1) if last else (0, 2)
    hx, hsx = h.reshape(x.shape), hs.reshape(x.shape)
    at = (lambda p: p[None, None, :]) if last else (lambda p: p[None, :, None])
    wf = 1.0 if w is None else at(w)
    q, _ = _grouped(gz * wf, groups, last)
    qs, _ = _grouped(gzs * abs(wf), groups, last)
    m1, m2 = q.sum(axes, keepdims=True) / n, (q * h).sum(axes, keepdims=True) / n
    s1, s2 = qs.sum(axes, keepdims=True) / n, (qs * hs).sum(axes, keepdims=True) / n
    gx = (r * (q - m1 - h * m2)).reshape(x.shape)
    gxs = (r * (qs + s1 + hs * s2 + hs * abs(m2))).reshape(x.shape)
    return ((gx, (gz * hx).sum(over), gz.sum(over)), (gxs, (gzs * hsx).sum(over), gzs.sum(over)))


# -------------------------------------------------------------- 4-bit floats

MX4_VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx4(rows):
    """(codes [n][nb][32], scale bytes [n][nb]) of rows [n][C]."""
    n, C = rows.shape
    nb = -(-C // 32)
    b = np.zeros((n, nb * 32))
    b[:, :C] = rows
    b = b.reshape(n, nb, 32)
    codes, scales = np.zeros(b.shape, np.uint8), np.zeros((n, nb), np.uint8)
    for i in range(n):
        for k in range(nb):
            big = np.max(np.abs(b[i, k]))
            if not np.isfinite(big):
                scales[i, k] = 255
                continue
            e = -127 if big == 0 else max(math.frexp(big)[1] - 3, -127)
            scales[i, k] = e + 127
            v = np.abs(b[i, k]) * 2.0 ** -float(e)
            near = np.abs(v[:, None] - MX4_VALUES[None, :])
            # the nearest, of two as near the one with the even index
            best = np.where(near == near.min(1, keepdims=True), np.arange(8) % 2, 2).argmin(1)
            codes[i, k] = best + 8 * np.signbit(b[i, k])
    return codes, scales


def mx4_values(codes, scales, C):
    v = MX4_VALUES[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (v * step[..., None]).reshape(len(codes), -1)[:, :C]


def mx4_rows(x):
    """The rows (b, p) of channels of a field [B][C][P] or tokens [B][C]."""
    return x if x.ndim == 2 else np.moveaxis(x, 1, 2).reshape(-1, x.shape[1])


def mx4_trip(x):
    """What a field [B][C][P] or tokens [B][C] keep in 4-bit floats."""
    rows = mx4_rows(x)
    v = mx4_values(*mx4(rows), rows.shape[1])
    return v if x.ndim == 2 else np.moveaxis(v.reshape(x.shape[0], x.shape[2], x.shape[1]), 2, 1)


def mx4_mix(x, A, bias, add, kind):
    """(y, sizes of its terms) of fields [B][C][P] at the values given (kept or not)."""
    z = np.einsum("oi,bip->bop", A, x)
    size = np.einsum("oi,bip->bop", abs(A), abs(x))
    for t in (None if bias is None else bias[None, :, None], add):
        if t is not None:
            z, size = z + t, size + abs(t)
    return (act(z, 1) if kind else z), size
