"""Binding of the training operators around a block (include/fno.h): 8-bit
activation checkpoints, the channel mix that keeps them with its backward, and
the norms with gate and residual scale. The names
are re-exported by the package; like the rest of the binding these functions
check and marshal arguments, every value is computed in the library's kernels.
"""

import ctypes
import functools

from ._lib import DTYPES, NORM_KINDS, SIGNATURES, NormGradsStruct, NormParamsStruct, check, lib

_NORM_NAMES = ("w_post", "b_post", "gate", "scale", "w_pre", "b_pre")

# A call on a small field takes a few microseconds on the GPU, so the checks on the
# way there are few: the extension (csrc/binding.cpp) looks at all of a call's tensors at
# once, and where one does not fit _ptr() or _buffer() find out what is wrong and say so.
_INT_MAX = (1 << 31) - 1
_torch = None
_names = None
_native = None
_functions = {}


def _t():
    """torch, imported on first use (importing the binding does not import it), and with it the extension."""
    global _torch, _names, _native
    if _torch is None:
        import torch
        try:
            from . import _native as native
        except ImportError as e:  # not there, or built against another torch
            raise RuntimeError(f"_native.so does not load: {e} (run python -m spectral_convolution_amd.build)") from e
        _names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
        _native, _torch = native, torch
    return _torch


def _refuse(name, t, shape, dtype, dev, optional):
    if not isinstance(t, _t().Tensor):
        raise TypeError(f"{name} must be a torch tensor" + (" or None" if optional else ""))
    if t.dtype != dtype:
        raise ValueError(f"{name} dtype {t.dtype} != {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call's first field on device {dev}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(name, t, shape, dtype, dev, optional=False):
    """Address of t, which has this shape and dtype, is contiguous and on device `dev`."""
    if t is None and optional:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, shape, dtype, dev, optional)


def _ptrs(names, need, td, dev, ref, *pairs):
    """Addresses of the tensors in pairs (tensor, shape, tensor, shape, ...), of ref's
    dtype td and device dev; the first `need` of them may not be None."""
    got = _native.addresses(ref, *pairs)
    if got is None or 0 in got[:need]:
        got = tuple(_ptr(n, t, s, td, dev, i >= need)
                    for i, (n, t, s) in enumerate(zip(names, pairs[::2], pairs[1::2])))
    return got


def _buffer(name, t, need, align, ref):
    """Address of a buffer of at least `need` bytes at a multiple of `align`, on ref's device."""
    try:
        p = _native.buffer(ref, t, need, align)
    except OverflowError:
        p = None
    if p is not None:
        return p
    if not isinstance(t, _t().Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    have = t.numel() * t.element_size()
    if have < need:
        raise ValueError(f"{name} holds {have} bytes, the call needs {need}")
    p = t.data_ptr()
    if p % align:
        raise ValueError(f"{name} must be {align}-byte aligned")
    if t.get_device() != ref.get_device() or not t.is_contiguous():
        _refuse(name, t, t.shape, t.dtype, ref.get_device(), False)
    return p


def _field(t, name):
    """(dtype name, dtype, device, shape as a tuple) of a field."""
    torch = _t()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    dt = _names.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} dtype {t.dtype} is not one of float32, float16, bfloat16")
    return dt, t.dtype, t.get_device(), tuple(t.shape)


def _split(shape, name):
    """(batch, channels, pixels) of [B][C](...)."""
    if len(shape) < 2:
        raise ValueError(f"{name} must be [batch][channels](...), got {shape}")
    P = 1
    for s in shape[2:]:
        P *= s
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:  # ctypes would pass on the low 32 bits
        raise ValueError(f"{name} shape {shape}: batch and channels must be below 2^31")
    return shape[0], shape[1], P


def _call(fn, dev, stream, *args):
    """Call the library with the tensors' device current, on `stream` or the current one."""
    torch = _t()
    if dev < 0:
        raise ValueError(f"{fn}: the tensors must be on the GPU")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    f = _functions.get(fn)
    if f is None:
        f = _functions[fn] = getattr(lib(), fn)
    st = f(*args, stream)
    if st:
        check(st, fn)


@functools.lru_cache(maxsize=1024)
def _bytes(fn, *args):
    """A size that the library computes from a shape (a call asks for the same ones every time)."""
    for v, t in zip(args, SIGNATURES[fn][1]):  # ctypes would pass on the low bits
        if t(v).value != v:
            raise ValueError(f"{fn}: {v} is out of the library's range")
    n = ctypes.c_size_t()
    check(getattr(lib(), fn)(*args, ctypes.byref(n)), fn)
    return n.value


def _empty(n, like):
    torch = _t()
    return torch.empty(n, dtype=torch.uint8, device=like.device)


# --------------------------------------------------------------- checkpoints

def _rows(shape):
    n = shape[-1] if shape else 1
    rows = 1
    for s in shape[:-1]:
        rows *= s
    return rows, n


def fno_checkpoint_bytes(rows, n):
    """Bytes of the 8-bit checkpoint of `rows` rows of n values."""
    return _bytes("fno_checkpoint_bytes", rows, n)


def fno_checkpoint_empty(x):
    """A device buffer (uint8 tensor) for the checkpoint of x (rows along its last axis)."""
    return _empty(fno_checkpoint_bytes(*_rows(tuple(x.shape))), x)


def fno_checkpoint_pack(x, saved, stream=None):
    """Keep x in 8 bits (blocks of 32 along its last axis) in `saved`."""
    dt, td, dev, shape = _field(x, "x")
    rows, n = _rows(shape)
    s = _buffer("saved", saved, fno_checkpoint_bytes(rows, n), 256, x)
    (p,) = _ptrs(("x",), 1, td, dev, x, x, shape)
    _call("fno_checkpoint_pack", dev, stream, p, s, rows, n, DTYPES[dt])


def fno_checkpoint_unpack(saved, y, stream=None):
    """Read the values kept in `saved` back into y (shape and dtype as packed)."""
    dt, td, dev, shape = _field(y, "y")
    rows, n = _rows(shape)
    s = _buffer("saved", saved, fno_checkpoint_bytes(rows, n), 256, y)
    (p,) = _ptrs(("y",), 1, td, dev, y, y, shape)
    _call("fno_checkpoint_unpack", dev, stream, s, p, rows, n, DTYPES[dt])


# --------------------------------------------------------------- channel mix

_MIX_FORWARD = ("x", "A", "y", "bias", "add")
_MIX_BACKWARD = ("A", "gy", "bias", "gx", "gA", "gbias", "gadd")


def fno_channel_mix_saved_bytes(batch, c_in, c_out, pixels, act=0, has_add=False):
    """Bytes of what fno_channel_mix_save keeps."""
    return _bytes("fno_channel_mix_saved_bytes", batch, c_in, c_out, pixels, act, int(has_add))


def fno_channel_mix_workspace_bytes(batch, c_in, c_out, pixels, dtype="f32"):
    """Bytes of the backward's workspace."""
    return _bytes("fno_channel_mix_workspace_bytes", batch, c_in, c_out, pixels, DTYPES[dtype])


def fno_channel_mix_saved_empty(x, c_out, act=0, has_add=False):
    """A device buffer (uint8 tensor) for what fno_channel_mix_save keeps."""
    B, I, P = _split(tuple(x.shape), "x")
    return _empty(fno_channel_mix_saved_bytes(B, I, c_out, P, act, has_add), x)


def fno_channel_mix_workspace_empty(x, c_out):
    """A device buffer (uint8 tensor) for the backward of a mix of x."""
    dt, _, _, shape = _field(x, "x")
    B, I, P = _split(shape, "x")
    return _empty(fno_channel_mix_workspace_bytes(B, I, c_out, P, dt), x)


def fno_channel_mix_save(x, A, bias, add, y, saved, act=0, stream=None):
    """fno_channel_mix that also keeps x (and, with GELU, add) in 8 bits in `saved`."""
    dt, td, dev, shape = _field(x, "x")
    B, I, P = _split(shape, "x")
    O = _split(_field(y, "y")[3], "y")[1]
    out = (B, O) + shape[2:]
    px, pA, py, pbias, padd = _ptrs(_MIX_FORWARD, 3, td, dev, x, x, shape, A, (O, I), y, out, bias, (O,), add, out)
    ps = _buffer("saved", saved, fno_channel_mix_saved_bytes(B, I, O, P, act, add is not None), 256, x)
    _call("fno_channel_mix_save", dev, stream, px, pA, pbias, padd, py, ps, B, I, O, P, act, DTYPES[dt])


def fno_channel_mix_backward_saved(saved, A, bias, gy, gx, gA, gbias, gadd, workspace, act=0, has_add=False,
                                   stream=None):
    """Gradients of the channel mix at what its forward kept: gx, gA, gbias,
    gadd, each None where not wanted. workspace: fno_channel_mix_workspace_empty."""
    dt, td, dev, shape = _field(gy, "gy")
    B, O, P = _split(shape, "gy")
    if not isinstance(A, _t().Tensor):
        raise TypeError("A must be a torch tensor")
    if A.dim() != 2 or A.shape[0] != O:
        raise ValueError(f"A shape {tuple(A.shape)} does not map to gy's {O} channels")
    I = A.shape[1]
    ps = _buffer("saved", saved, fno_channel_mix_saved_bytes(B, I, O, P, act, has_add), 256, gy)
    pA, pgy, pbias, pgx, pgA, pgbias, pgadd = _ptrs(_MIX_BACKWARD, 2, td, dev, gy, A, (O, I), gy, shape, bias, (O,), gx,
                                                    (B, I) + shape[2:], gA, (O, I), gbias, (O,), gadd, shape)
    ws = None
    if gA is not None or gbias is not None:
        ws = _buffer("workspace", workspace, fno_channel_mix_workspace_bytes(B, I, O, P, dt), 16, gy)
    _call("fno_channel_mix_backward_saved", dev, stream, ps, pA, pbias, pgy, pgx, pgA, pgbias, pgadd, ws, B, I, O, P,
          act, int(has_add), DTYPES[dt])


# --------------------------------------------------------------------- norms

class NormParams:
    """Parameters of the norms around a block: kind "rms" or "layer", eps, and
    w_post, b_post, scale, w_pre, b_pre [C] and gate [B][C], each a tensor or
    None (weights, gate and scale then count as 1, biases as 0)."""

    __slots__ = ("kind", "eps") + _NORM_NAMES

    def __init__(self, kind, eps, w_post=None, b_post=None, gate=None, scale=None, w_pre=None, b_pre=None):
        if kind not in NORM_KINDS:
            raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}")
        self.kind, self.eps = kind, eps
        self.w_post, self.b_post, self.gate, self.scale = w_post, b_post, gate, scale
        self.w_pre, self.b_pre = w_pre, b_pre

    def _pairs(self, B, C):
        c = (C,)
        return self.w_post, c, self.b_post, c, self.gate, (B, C), self.scale, c, self.w_pre, c, self.b_pre, c

    def _struct(self, addresses):
        return NormParamsStruct(NORM_KINDS[self.kind], self.eps, *addresses)


class NormGrads:
    """Where the gradients of the parameters go; None: not wanted."""

    __slots__ = _NORM_NAMES

    def __init__(self, w_post=None, b_post=None, gate=None, scale=None, w_pre=None, b_pre=None):
        self.w_post, self.b_post, self.gate, self.scale = w_post, b_post, gate, scale
        self.w_pre, self.b_pre = w_pre, b_pre

    _pairs = NormParams._pairs


def fno_norm_residual_saved_bytes(batch, channels, pixels):
    """Bytes of the checkpoints fno_norm_residual_save leaves."""
    return _bytes("fno_norm_residual_saved_bytes", batch, channels, pixels)


def fno_norm_residual_workspace_bytes(batch, channels, pixels, dtype="f32"):
    """Bytes of the backward's workspace."""
    return _bytes("fno_norm_residual_workspace_bytes", batch, channels, pixels, DTYPES[dtype])


def fno_norm_residual_saved_empty(x):
    """A device buffer (uint8 tensor) for the checkpoints of a field or of tokens shaped like x."""
    return _empty(fno_norm_residual_saved_bytes(*_split(tuple(x.shape), "x")), x)


def fno_norm_residual_workspace_empty(x):
    """A device buffer (uint8 tensor) for the backward of a call on x."""
    dt, _, _, shape = _field(x, "x")
    return _empty(fno_norm_residual_workspace_bytes(*_split(shape, "x"), dt), x)


_NORM_FORWARD = ("x", "v", "y", "u") + _NORM_NAMES
_NORM_BACKWARD = (("gy", "x", "v", "gu", "gx", "gv") + _NORM_NAMES + tuple("gradient of " + n for n in _NORM_NAMES))
_NORM_BACKWARD_SAVED = _NORM_BACKWARD[:1] + _NORM_BACKWARD[3:]


def _norm_forward(fn, prm, x, v, y, u, saved, stream):
    dt, td, dev, shape = _field(x, "x")
    B, C, P = _split(shape, "x")
    p = _ptrs(_NORM_FORWARD, 3, td, dev, x, x, shape, v, shape, y, shape, u, shape, *prm._pairs(B, C))
    args = p[:4]
    if saved is not False:
        args += (_buffer("saved", saved, fno_norm_residual_saved_bytes(B, C, P), 256, x),)
    _call(fn, dev, stream, prm._struct(p[4:]), *args, B, C, P, DTYPES[dt])


def fno_norm_residual(params, x, v, y, u, stream=None):
    """y = x + scale gate N_post(v), u = N_pre(y) over the channels of
    [B][C](...) fields or [B][C] tokens; u may be None."""
    _norm_forward("fno_norm_residual", params, x, v, y, u, False, stream)


def fno_norm_residual_save(params, x, v, y, u, saved, stream=None):
    """fno_norm_residual that also keeps x and v in 8 bits in `saved`."""
    _norm_forward("fno_norm_residual_save", params, x, v, y, u, saved, stream)


def _norm_backward(fn, prm, x, v, saved, gy, gu, gx, gv, grads, workspace, stream):
    dt, td, dev, shape = _field(gy, "gy")
    B, C, P = _split(shape, "gy")
    tail = (gu, shape, gx, shape, gv, shape) + prm._pairs(B, C)
    if grads is not None:
        tail += grads._pairs(B, C)
    if saved is False:
        p = _ptrs(_NORM_BACKWARD, 3, td, dev, gy, gy, shape, x, shape, v, shape, *tail)
        first, p = p[1:3], p[:1] + p[3:]
    else:
        p = _ptrs(_NORM_BACKWARD_SAVED, 1, td, dev, gy, gy, shape, *tail)
        first = (_buffer("saved", saved, fno_norm_residual_saved_bytes(B, C, P), 256, gy),)
    wanted = p[10:]
    ws = None
    if any(wanted):
        ws = _buffer("workspace", workspace, fno_norm_residual_workspace_bytes(B, C, P, dt), 16, gy)
    _call(fn, dev, stream, prm._struct(p[4:10]), *first, *p[:4], NormGradsStruct(*wanted), ws, B, C, P, DTYPES[dt])


def fno_norm_residual_backward(params, x, v, gy, gu, gx, gv, grads, workspace, stream=None):
    """Gradients of fno_norm_residual at gy = dL/dy, gu = dL/du (None: none
    through u): gx, gv (None: not wanted) and those named in grads (NormGrads or
    None). workspace: fno_norm_residual_workspace_empty."""
    _norm_backward("fno_norm_residual_backward", params, x, v, False, gy, gu, gx, gv, grads, workspace, stream)


def fno_norm_residual_backward_saved(params, saved, gy, gu, gx, gv, grads, workspace, stream=None):
    """fno_norm_residual_backward at the x and v read back from `saved`."""
    _norm_backward("fno_norm_residual_backward_saved", params, None, None, saved, gy, gu, gx, gv, grads, workspace,
                   stream)


# ------------------------------------------------- differentiable functions

def channel_mix(x, A, bias=None, add=None, act=0):
    """y = act(A x + bias + add), differentiable in all four; x (and, with
    GELU, add) is kept for the backward in 8 bits, rows along the pixels (33
    bytes for each 32 of them: fields of a few pixels take more than they have).
    Without gradients the same kernel runs and what it kept is dropped: y is the
    same either way, and fno_channel_mix, which keeps nothing, is mostly slower, and at best 0.8 of it (16-bit fields of up to 64 channels)."""
    from ._training_autograd import ChannelMixFunction
    if not isinstance(A, _t().Tensor) or A.dim() != 2:
        raise ValueError("A must be a [c_out][c_in] tensor")
    return ChannelMixFunction.apply(x, A, bias, add, act)


def norm_residual(x, v, params, with_u=True, keep="8bit"):
    """(y, u) of fno_norm_residual (u None unless with_u), differentiable in x, v
    and the parameters (NormParams); x and v are kept for the backward in 8 bits
    (keep "8bit") or as they are ("whole"), where one is wanted."""
    from ._training_autograd import NormResidualFunction
    if keep not in ("8bit", "whole"):
        raise ValueError('keep must be "8bit" or "whole"')
    prm = [getattr(params, k) for k in _NORM_NAMES]
    torch = _t()
    if not torch.is_grad_enabled() or not any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, v, *prm)):
        keep = "whole"  # no backward follows: no checkpoints are written, and whole fields are not held either
    return NormResidualFunction.apply(x, v, params.kind, params.eps, keep, with_u, *prm)
