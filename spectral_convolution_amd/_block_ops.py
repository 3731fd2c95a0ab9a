"""Binding of the operators of a regularised block (include/fno.h): group norm
with an activation and dropout, dropout into a residual stream, and the block's channel
mix on microscaled 4-bit floats, for serving. The names are
re-exported by the package; these functions check and marshal arguments, every
value is computed in the library's kernels.
"""

import functools

from . import _training as base
from ._lib import DROP_UNITS, DTYPES, DropoutStruct, GroupNormParamsStruct

_U64 = 1 << 64
_I64 = (1 << 63) - 1


def _split(shape, name, last):
    """(batch, channels, pixels) of [B][C](...), or of [B](...)[C] where last."""
    if not last:
        return base._split(shape, name)
    if len(shape) < 2:
        raise ValueError(f"{name} must be [batch](...)[channels], got {shape}")
    B, C, P = base._split((shape[0], shape[-1]) + shape[1:-1], name)
    return B, C, P


# ------------------------------------------------------------------- dropout

class Dropout:
    """What a call drops: units ("element", "channel" of a sample, "sample") with
    probability p (to 1/65536), by the random bits that belong to seed and offset
    (each below 2^64). A program moves the offset on with every call; a backward takes
    the forward's. An object does not change: a backward finds what its forward had. step: a device int64 tensor of one value that is added to the offset when the
    call runs, for captured graphs (not to be moved on between a forward and its backward)."""

    __slots__ = ("p", "seed", "offset", "unit", "step", "_s")

    def __init__(self, p, seed, offset=0, unit="element", step=None):
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p must be in [0, 1], got {p}")
        if unit not in DROP_UNITS:
            raise ValueError(f"unit must be one of {list(DROP_UNITS)}")
        for name, v in (("seed", seed), ("offset", offset)):
            if not 0 <= v < _U64:
                raise ValueError(f"{name} must be in [0, 2^64), got {v}")
        if step is not None:
            torch = base._t()
            if not isinstance(step, torch.Tensor) or step.dtype != torch.int64 or step.numel() != 1:
                raise ValueError("step must be an int64 tensor of one value")
        for name, v in zip(self.__slots__, (p, seed, offset, unit, step, DropoutStruct(p, DROP_UNITS[unit], seed, offset, None))):
            object.__setattr__(self, name, v)

    def __setattr__(self, name, value):
        raise AttributeError(f"a Dropout does not change: make another for another {name}")

    def __reduce__(self):
        return Dropout, (self.p, self.seed, self.offset, self.unit, self.step)

    def _struct(self, ref):
        """fno_dropout_t for a call on ref's device."""
        if self.step is not None:
            self._s.step = base._buffer("step", self.step, 8, 8, ref)
        return self._s


def _drop(dropout, ref):
    if dropout is None:
        return None
    if not isinstance(dropout, Dropout):
        raise TypeError("dropout must be a Dropout or None")
    return dropout._struct(ref)


def fno_dropout_residual(dropout, x, v, y, channels_last=False, stream=None):
    """y = x + D(v) (x None: y = D(v)) on [B][C](...) or [B](...)[C] fields; also the
    backward of both, on dL/dy with x None."""
    dt, td, dev, shape = base._field(v, "v")
    B, C, P = _split(shape, "v", channels_last)
    if dropout is None:
        raise TypeError("dropout must be a Dropout")
    pv, py, px = base._ptrs(("v", "y", "x"), 2, td, dev, v, v, shape, y, shape, x, shape)
    base._call("fno_dropout_residual", dev, stream, _drop(dropout, v), px, pv, py, B, C, P, int(channels_last), DTYPES[dt])


# ---------------------------------------------------------------- group norm

class GroupNormParams:
    """A group norm: the number of groups, eps, weight and bias [C] (tensors or None: 1
    and 0), act (0: none, 1: GELU, 2: SiLU), and whether fields have their channels last."""

    __slots__ = ("groups", "eps", "weight", "bias", "act", "channels_last")

    def __init__(self, groups, eps=1e-5, weight=None, bias=None, act=0, channels_last=False):
        if act not in (0, 1, 2):
            raise ValueError("act must be 0 (none), 1 (GELU) or 2 (SiLU)")
        if not 0 < groups <= base._INT_MAX:
            raise ValueError(f"groups must be positive, got {groups}")
        self.groups, self.eps, self.weight, self.bias = groups, eps, weight, bias
        self.act, self.channels_last = act, bool(channels_last)

    def _struct(self, weight, bias):
        return GroupNormParamsStruct(self.groups, self.act, int(self.channels_last), self.eps, weight, bias)


def fno_group_norm_workspace_bytes(batch, channels, pixels, groups, channels_last=False, dtype="f32"):
    """Bytes of the workspace of either call."""
    return base._bytes("fno_group_norm_workspace_bytes", batch, channels, pixels, groups, int(channels_last), DTYPES[dtype])


def fno_group_norm_workspace_empty(x, groups, channels_last=False):
    """A device buffer (uint8 tensor) for the calls on fields shaped like x."""
    dt, _, _, shape = base._field(x, "x")
    return base._empty(fno_group_norm_workspace_bytes(*_split(shape, "x", channels_last), groups, channels_last, dt), x)


def fno_group_norm_stats_empty(x, groups):
    """A float32 tensor [B][groups][2] for the statistics of x's groups."""
    torch = base._t()
    return torch.empty((x.shape[0], groups, 2), dtype=torch.float32, device=x.device)


@functools.lru_cache(maxsize=1)
def _f32():
    return base._t().float32


def _stats(stats, B, G, dev, optional):
    return base._ptr("stats", stats, (B, G, 2), _f32(), dev, optional)


def fno_group_norm(params, x, y, stats, workspace, dropout=None, stream=None):
    """y = D(act(group norm of x)); stats (float32 [B][groups][2] or None) takes what the
    backward needs. workspace: fno_group_norm_workspace_empty."""
    dt, td, dev, shape = base._field(x, "x")
    last, G = params.channels_last, params.groups
    B, C, P = _split(shape, "x", last)
    c = (C,)
    px, py, pw, pb = base._ptrs(("x", "y", "weight", "bias"), 2, td, dev, x, x, shape, y, shape, params.weight, c,
                                params.bias, c)
    ws = base._buffer("workspace", workspace, fno_group_norm_workspace_bytes(B, C, P, G, last, dt), 16, x)
    ps = _stats(stats, B, G, dev, True)
    base._call("fno_group_norm", dev, stream, params._struct(pw, pb), _drop(dropout, x), px, py, ps, ws, B, C, P, DTYPES[dt])


def fno_group_norm_backward(params, x, stats, gy, gx, gw, gb, workspace, dropout=None, stream=None):
    """Gradients of fno_group_norm at gy = dL/dy, with the forward's x, stats and dropout: gx, gw, gb
    (of weight and bias), each None where not wanted."""
    dt, td, dev, shape = base._field(x, "x")
    last, G = params.channels_last, params.groups
    B, C, P = _split(shape, "x", last)
    c = (C,)
    px, pgy, pw, pb, pgx, pgw, pgb = base._ptrs(("x", "gy", "weight", "bias", "gx", "gw", "gb"), 2, td, dev, x, x, shape,
                                                gy, shape, params.weight, c, params.bias, c, gx, shape, gw, c, gb, c)
    ws = base._buffer("workspace", workspace, fno_group_norm_workspace_bytes(B, C, P, G, last, dt), 16, x)
    ps = _stats(stats, B, G, dev, False)
    base._call("fno_group_norm_backward", dev, stream, params._struct(pw, pb), _drop(dropout, x), px, ps, pgy, pgx, pgw,
               pgb, ws, B, C, P, DTYPES[dt])


# -------------------------------------------------------------- 4-bit floats

def fno_mx4_bytes(batch, channels, pixels=1):
    """Bytes of a [batch][channels][pixels] field (a weight: [c_out][c_in]) in 4-bit floats."""
    return base._bytes("fno_mx4_bytes", batch, channels, pixels)


def fno_mx4_empty(x):
    """A device buffer (uint8 tensor) for x, [B][C](...), in 4-bit floats."""
    return base._empty(fno_mx4_bytes(*base._split(tuple(x.shape), "x")), x)


def fno_mx4_pack(x, packed, stream=None):
    """Keep x, [B][C](...), in 4-bit floats in `packed`: blocks of 32 along the channels."""
    dt, td, dev, shape = base._field(x, "x")
    B, C, P = base._split(shape, "x")
    s = base._buffer("packed", packed, fno_mx4_bytes(B, C, P), 256, x)
    (p,) = base._ptrs(("x",), 1, td, dev, x, x, shape)
    base._call("fno_mx4_pack", dev, stream, p, s, B, C, P, DTYPES[dt])


def fno_mx4_unpack(packed, y, stream=None):
    """Read the values kept in `packed` back into y (shape as packed)."""
    dt, td, dev, shape = base._field(y, "y")
    B, C, P = base._split(shape, "y")
    s = base._buffer("packed", packed, fno_mx4_bytes(B, C, P), 256, y)
    (p,) = base._ptrs(("y",), 1, td, dev, y, y, shape)
    base._call("fno_mx4_unpack", dev, stream, s, p, B, C, P, DTYPES[dt])


def fno_channel_mix_mx4(xq, Aq, bias, add, y, c_in, act=0, stream=None):
    """y = act(A x + bias + add) of a packed field (or tokens) of c_in channels and a packed weight; y
    [B][c_out](...), bias and add (either may be None) have the storage type."""
    dt, td, dev, shape = base._field(y, "y")
    B, O, P = base._split(shape, "y")
    py, pbias, padd = base._ptrs(("y", "bias", "add"), 1, td, dev, y, y, shape, bias, (O,), add, shape)
    px = base._buffer("xq", xq, fno_mx4_bytes(B, c_in, P), 256, y)
    pA = base._buffer("Aq", Aq, fno_mx4_bytes(O, c_in), 256, y)
    base._call("fno_channel_mix_mx4", dev, stream, px, pA, pbias, padd, py, B, c_in, O, P, act, DTYPES[dt])


class Mx4Weight:
    """A weight [c_out][c_in] kept in 4-bit floats for channel_mix_mx4: 17 bytes for each 32 values that
    a row begins."""

    __slots__ = ("c_out", "c_in", "packed")

    def __init__(self, A):
        torch = base._t()
        if not isinstance(A, torch.Tensor) or A.dim() != 2:
            raise ValueError("A must be a [c_out][c_in] tensor")
        A = A.detach().contiguous()
        if A.data_ptr() % 16:
            A = A.clone()
        self.c_out, self.c_in = A.shape
        self.packed = fno_mx4_empty(A)
        fno_mx4_pack(A, self.packed)


def channel_mix_mx4(x, weight, bias=None, add=None, act=0):
    """act(A x + bias + add) with A an Mx4Weight and x, [B][C](...), packed to 4-bit floats on the
    way. For serving: it has no gradient, and refuses inputs that want one."""
    torch = base._t()
    if not isinstance(weight, Mx4Weight):
        raise TypeError("weight must be an Mx4Weight")
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, bias, add)):
        raise ValueError("channel_mix_mx4 has no gradient: call it under torch.no_grad()")
    from ._training_autograd import _dense
    x, add = _dense(x), _dense(add)
    shape = tuple(x.shape)
    if len(shape) < 2 or shape[1] != weight.c_in:
        raise ValueError(f"x shape {shape} does not have the weight's {weight.c_in} channels")
    packed = fno_mx4_empty(x)
    fno_mx4_pack(x, packed)
    y = torch.empty((shape[0], weight.c_out) + shape[2:], dtype=x.dtype, device=x.device)
    fno_channel_mix_mx4(packed, weight.packed, None if bias is None else bias.contiguous(), add, y, weight.c_in, act)
    return y


# ------------------------------------------------- differentiable functions

def group_norm(x, params, dropout=None):
    """D(act(group norm of x)), differentiable in x, params.weight and params.bias; x and
    the groups' statistics are kept for the backward, no mask is. A call captured into a graph
    whose leaves an autograd graph on another stream holds is refused; under torch.no_grad() it is not."""
    from ._block_autograd import GroupNormFunction
    from ._capture import check_call
    check_call(x, params.weight, params.bias)
    return GroupNormFunction.apply(x, params.weight, params.bias, params, dropout)


def dropout_residual(v, dropout, x=None, channels_last=False):
    """x + D(v) (x None: D(v)), differentiable in both; nothing is kept for the backward.
    Captured calls: as group_norm."""
    from ._block_autograd import DropoutResidualFunction
    from ._capture import check_call
    check_call(v, x)
    return DropoutResidualFunction.apply(v, x, dropout, channels_last)
