"""Binding of the training operators around a block (include/fno.h): 8-bit
activation checkpoints, the channel mix that keeps them with its backward, and
the norms with gate and residual scale. The names
are re-exported by the package; like the rest of the binding these functions
check and marshal arguments, every value is computed in the library's kernels.
"""

import ctypes

from ._lib import DTYPES, NORM_KINDS, NormGradsStruct, NormParamsStruct, check, lib

_NORM_NAMES = ("w_post", "b_post", "gate", "scale", "w_pre", "b_pre")


def _field_dtype(t, name):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    if t.dtype not in names:
        raise ValueError(f"{name} dtype {t.dtype} is not one of float32, float16, bfloat16")
    return names[t.dtype]


def _check(name, t, shape, like, optional=False):
    """t has `shape` and lives in like's dtype and device."""
    import torch
    if t is None:
        if optional:
            return
        raise TypeError(f"{name} must be a torch tensor")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor" + (" or None" if optional else ""))
    if t.dtype != like.dtype:
        raise ValueError(f"{name} dtype {t.dtype} != {like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name} is on {t.device}, not on {like.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")


def _check_buffer(name, t, need, align, device):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    have = t.numel() * t.element_size()
    if have < need:
        raise ValueError(f"{name} holds {have} bytes, the call needs {need}")
    if t.data_ptr() % align:
        raise ValueError(f"{name} must be {align}-byte aligned")


def _ptr(t):
    from . import _ptr as ptr
    return ptr(t)


def _stream(stream, like):
    from . import _stream as s
    return s(stream, like.device)


def _bytes(fn, *args):
    n = ctypes.c_size_t()
    check(getattr(lib(), fn)(*args, ctypes.byref(n)), fn)
    return n.value


class _on:
    """The tensor's device as the current one, where the library launches."""

    def __init__(self, t):
        self.t = t

    def __enter__(self):
        import torch
        self.guard = torch.cuda.device(self.t.device)
        return self.guard.__enter__()

    def __exit__(self, *a):
        return self.guard.__exit__(*a)


# --------------------------------------------------------------- checkpoints

def _rows(t):
    n = t.shape[-1] if t.dim() else 1
    return (t.numel() // n if n else 0), n


def fno_checkpoint_bytes(rows, n):
    """Bytes of the 8-bit checkpoint of `rows` rows of n values."""
    return _bytes("fno_checkpoint_bytes", rows, n)


def fno_checkpoint_empty(x):
    """A device buffer (uint8 tensor) for the checkpoint of x (rows along its last axis)."""
    import torch
    return torch.empty(fno_checkpoint_bytes(*_rows(x)), dtype=torch.uint8, device=x.device)


def fno_checkpoint_pack(x, saved, stream=None):
    """Keep x in 8 bits (blocks of 32 along its last axis) in `saved`."""
    dt = _field_dtype(x, "x")
    rows, n = _rows(x)
    _check_buffer("saved", saved, fno_checkpoint_bytes(rows, n), 256, x.device)
    with _on(x):
        check(lib().fno_checkpoint_pack(_ptr(x), _ptr(saved), rows, n, DTYPES[dt], _stream(stream, x)),
              "fno_checkpoint_pack")


def fno_checkpoint_unpack(saved, y, stream=None):
    """Read the values kept in `saved` back into y (shape and dtype as packed)."""
    dt = _field_dtype(y, "y")
    rows, n = _rows(y)
    _check_buffer("saved", saved, fno_checkpoint_bytes(rows, n), 256, y.device)
    with _on(y):
        check(lib().fno_checkpoint_unpack(_ptr(saved), _ptr(y), rows, n, DTYPES[dt], _stream(stream, y)),
              "fno_checkpoint_unpack")


# --------------------------------------------------------------- channel mix

def _fold(t, name):
    """(dtype, batch, channels, pixels) of [B][C](...)."""
    dt = _field_dtype(t, name)
    if t.dim() < 2:
        raise ValueError(f"{name} must be [batch][channels](...), got {tuple(t.shape)}")
    P = 1
    for s in t.shape[2:]:
        P *= s
    return dt, t.shape[0], t.shape[1], P


def fno_channel_mix_saved_bytes(batch, c_in, c_out, pixels, act=0, has_add=False):
    """Bytes of what fno_channel_mix_save keeps."""
    return _bytes("fno_channel_mix_saved_bytes", batch, c_in, c_out, pixels, act, int(has_add))


def fno_channel_mix_workspace_bytes(batch, c_in, c_out, pixels, dtype="f32"):
    """Bytes of the backward's workspace."""
    return _bytes("fno_channel_mix_workspace_bytes", batch, c_in, c_out, pixels, DTYPES[dtype])


def fno_channel_mix_saved_empty(x, c_out, act=0, has_add=False):
    """A device buffer (uint8 tensor) for what fno_channel_mix_save keeps."""
    import torch
    _, B, I, P = _fold(x, "x")
    return torch.empty(fno_channel_mix_saved_bytes(B, I, c_out, P, act, has_add), dtype=torch.uint8, device=x.device)


def fno_channel_mix_workspace_empty(x, c_out):
    """A device buffer (uint8 tensor) for the backward of a mix of x."""
    import torch
    dt, B, I, P = _fold(x, "x")
    return torch.empty(fno_channel_mix_workspace_bytes(B, I, c_out, P, dt), dtype=torch.uint8, device=x.device)


def fno_channel_mix_save(x, A, bias, add, y, saved, act=0, stream=None):
    """fno_channel_mix that also keeps x (and, with GELU, add) in 8 bits in `saved`."""
    dt, B, I, P = _fold(x, "x")
    _, By, O, Py = _fold(y, "y")
    _check("y", y, (B, O) + tuple(x.shape[2:]), x)
    _check("A", A, (O, I), x)
    _check("bias", bias, (O,), x, optional=True)
    _check("add", add, y.shape, x, optional=True)
    _check_buffer("saved", saved, fno_channel_mix_saved_bytes(B, I, O, P, act, add is not None), 256, x.device)
    with _on(x):
        check(lib().fno_channel_mix_save(_ptr(x), _ptr(A), _ptr(bias), _ptr(add), _ptr(y), _ptr(saved), B, I, O, P, act,
                                         DTYPES[dt], _stream(stream, x)), "fno_channel_mix_save")


def fno_channel_mix_backward_saved(saved, A, bias, gy, gx, gA, gbias, gadd, workspace, act=0, has_add=False,
                                   stream=None):
    """Gradients of the channel mix at what its forward kept: gx, gA, gbias,
    gadd, each None where not wanted. workspace: fno_channel_mix_workspace_empty."""
    dt, B, O, P = _fold(gy, "gy")
    if A.dim() != 2 or A.shape[0] != O:
        raise ValueError(f"A shape {tuple(A.shape)} does not map to gy's {O} channels")
    I = A.shape[1]
    _check("A", A, (O, I), gy)
    _check("bias", bias, (O,), gy, optional=True)
    _check("gx", gx, (B, I) + tuple(gy.shape[2:]), gy, optional=True)
    _check("gA", gA, (O, I), gy, optional=True)
    _check("gbias", gbias, (O,), gy, optional=True)
    _check("gadd", gadd, gy.shape, gy, optional=True)
    _check_buffer("saved", saved, fno_channel_mix_saved_bytes(B, I, O, P, act, has_add), 256, gy.device)
    if gA is not None or gbias is not None:
        _check_buffer("workspace", workspace, fno_channel_mix_workspace_bytes(B, I, O, P, dt), 16, gy.device)
    with _on(gy):
        check(lib().fno_channel_mix_backward_saved(_ptr(saved), _ptr(A), _ptr(bias), _ptr(gy), _ptr(gx), _ptr(gA),
                                                   _ptr(gbias), _ptr(gadd), _ptr(workspace), B, I, O, P, act,
                                                   int(has_add), DTYPES[dt], _stream(stream, gy)),
              "fno_channel_mix_backward_saved")


# --------------------------------------------------------------------- norms

class NormParams:
    """Parameters of the norms around a block: kind "rms" or "layer", eps, and
    w_post, b_post, scale, w_pre, b_pre [C] and gate [B][C], each a tensor or
    None (weights, gate and scale then count as 1, biases as 0)."""

    def __init__(self, kind, eps, w_post=None, b_post=None, gate=None, scale=None, w_pre=None, b_pre=None):
        if kind not in NORM_KINDS:
            raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}")
        self.kind, self.eps = kind, float(eps)
        self.w_post, self.b_post, self.gate, self.scale = w_post, b_post, gate, scale
        self.w_pre, self.b_pre = w_pre, b_pre


class NormGrads:
    """Where the gradients of the parameters go; None: not wanted."""

    def __init__(self, w_post=None, b_post=None, gate=None, scale=None, w_pre=None, b_pre=None):
        self.w_post, self.b_post, self.gate, self.scale = w_post, b_post, gate, scale
        self.w_pre, self.b_pre = w_pre, b_pre


def _norm_struct(obj, cls, like, B, C):
    shapes = {n: (B, C) if n == "gate" else (C,) for n in _NORM_NAMES}
    for n in _NORM_NAMES:
        _check(n if cls is NormParamsStruct else f"gradient of {n}", getattr(obj, n), shapes[n], like, optional=True)
    ptrs = {n: _ptr(getattr(obj, n)) for n in _NORM_NAMES}
    if cls is NormParamsStruct:
        return cls(NORM_KINDS[obj.kind], obj.eps, **ptrs)
    return cls(**ptrs)


def fno_norm_residual_saved_bytes(batch, channels, pixels):
    """Bytes of the checkpoints fno_norm_residual_save leaves."""
    return _bytes("fno_norm_residual_saved_bytes", batch, channels, pixels)


def fno_norm_residual_workspace_bytes(batch, channels, pixels, dtype="f32"):
    """Bytes of the backward's workspace."""
    return _bytes("fno_norm_residual_workspace_bytes", batch, channels, pixels, DTYPES[dtype])


def fno_norm_residual_saved_empty(x):
    """A device buffer (uint8 tensor) for the checkpoints of a field or of tokens shaped like x."""
    import torch
    _, B, C, P = _fold(x, "x")
    return torch.empty(fno_norm_residual_saved_bytes(B, C, P), dtype=torch.uint8, device=x.device)


def fno_norm_residual_workspace_empty(x):
    """A device buffer (uint8 tensor) for the backward of a call on x."""
    import torch
    dt, B, C, P = _fold(x, "x")
    return torch.empty(fno_norm_residual_workspace_bytes(B, C, P, dt), dtype=torch.uint8, device=x.device)


def _norm_forward(fn, prm, x, v, y, u, saved, stream):
    dt, B, C, P = _fold(x, "x")
    _check("v", v, x.shape, x)
    _check("y", y, x.shape, x)
    _check("u", u, x.shape, x, optional=True)
    st = _norm_struct(prm, NormParamsStruct, x, B, C)
    args = [_ptr(x), _ptr(v), _ptr(y), _ptr(u)]
    if fn == "fno_norm_residual_save":
        _check_buffer("saved", saved, fno_norm_residual_saved_bytes(B, C, P), 256, x.device)
        args.append(_ptr(saved))
    with _on(x):
        check(getattr(lib(), fn)(ctypes.byref(st), *args, B, C, P, DTYPES[dt], _stream(stream, x)), fn)


def fno_norm_residual(params, x, v, y, u, stream=None):
    """y = x + scale gate N_post(v), u = N_pre(y) over the channels of
    [B][C](...) fields or [B][C] tokens; u may be None."""
    _norm_forward("fno_norm_residual", params, x, v, y, u, None, stream)


def fno_norm_residual_save(params, x, v, y, u, saved, stream=None):
    """fno_norm_residual that also keeps x and v in 8 bits in `saved`."""
    _norm_forward("fno_norm_residual_save", params, x, v, y, u, saved, stream)


def _norm_backward(fn, prm, first, gy, gu, gx, gv, grads, workspace, stream):
    dt, B, C, P = _fold(gy, "gy")
    grads = NormGrads() if grads is None else grads
    for name, t in (("gu", gu), ("gx", gx), ("gv", gv)):
        _check(name, t, gy.shape, gy, optional=True)
    st = _norm_struct(prm, NormParamsStruct, gy, B, C)
    gr = _norm_struct(grads, NormGradsStruct, gy, B, C)
    if any(getattr(grads, n) is not None for n in _NORM_NAMES):
        _check_buffer("workspace", workspace, fno_norm_residual_workspace_bytes(B, C, P, dt), 16, gy.device)
    if fn == "fno_norm_residual_backward":
        for name, t in zip("xv", first):
            _check(name, t, gy.shape, gy)
    else:
        _check_buffer("saved", first[0], fno_norm_residual_saved_bytes(B, C, P), 256, gy.device)
    with _on(gy):
        check(getattr(lib(), fn)(ctypes.byref(st), *(_ptr(t) for t in first), _ptr(gy), _ptr(gu), _ptr(gx), _ptr(gv),
                                 ctypes.byref(gr), _ptr(workspace), B, C, P, DTYPES[dt], _stream(stream, gy)), fn)


def fno_norm_residual_backward(params, x, v, gy, gu, gx, gv, grads, workspace, stream=None):
    """Gradients of fno_norm_residual at gy = dL/dy, gu = dL/du (None: none
    through u): gx, gv (None: not wanted) and those named in grads (NormGrads or
    None). workspace: fno_norm_residual_workspace_empty."""
    _norm_backward("fno_norm_residual_backward", params, (x, v), gy, gu, gx, gv, grads, workspace, stream)


def fno_norm_residual_backward_saved(params, saved, gy, gu, gx, gv, grads, workspace, stream=None):
    """fno_norm_residual_backward at the x and v read back from `saved`."""
    _norm_backward("fno_norm_residual_backward_saved", params, (saved,), gy, gu, gx, gv, grads, workspace, stream)
