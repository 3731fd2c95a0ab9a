"""The training operators around a block as PyTorch autograd Functions: the
channel mix that keeps its inputs in 8 bits, and the norms with gate and residual
scale (fields kept in 8 bits or whole). Imported on first use, since it imports torch.
Every value is computed in the library's kernels; torch allocates the tensors."""

import torch
from torch.autograd.function import once_differentiable

from . import _training as ops


def _dense(t):
    """t as the kernels take a field: contiguous, on a 16-byte boundary."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"fields must be on the GPU, got one on {t.device}")
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class ChannelMixFunction(torch.autograd.Function):
    """y = act(A x + bias + add). Between forward and backward only the 8-bit
    checkpoints of x (and, with GELU, of add) and the weights live."""

    @staticmethod
    def forward(ctx, x, A, bias, add, act):
        x, add, A = _dense(x), _dense(add), A.contiguous()
        bias = None if bias is None else bias.contiguous()
        y = torch.empty((x.shape[0], A.shape[0]) + tuple(x.shape[2:]), dtype=x.dtype, device=x.device)
        saved = ops.fno_channel_mix_saved_empty(x, A.shape[0], act, add is not None)
        ops.fno_channel_mix_save(x, A, bias, add, y, saved, act)
        ctx.act, ctx.has_add, ctx.x_shape = act, add is not None, x.shape
        ctx.save_for_backward(saved, A, bias)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        saved, A, bias = ctx.saved_tensors
        need = ctx.needs_input_grad
        if not any(need[:4]):
            return None, None, None, None, None
        gy = _dense(gy)
        gx = torch.empty(ctx.x_shape, dtype=gy.dtype, device=gy.device) if need[0] else None
        gA = torch.empty_like(A) if need[1] else None
        gbias = torch.empty_like(bias) if need[2] else None
        gadd = torch.empty_like(gy) if need[3] else None
        ws = None
        if gA is not None or gbias is not None:
            B, I, P = ops._split(tuple(ctx.x_shape), "x")
            ws = ops._empty(ops.fno_channel_mix_workspace_bytes(B, I, A.shape[0], P, ops._field(gy, "gy")[0]), gy)
        ops.fno_channel_mix_backward_saved(saved, A, bias, gy, gx, gA, gbias, gadd, ws, ctx.act, ctx.has_add)
        return gx, gA, gbias, gadd, None


class NormResidualFunction(torch.autograd.Function):
    """(y, u) of fno_norm_residual. keep "8bit": the checkpoints of x and v live
    between forward and backward, "whole": x and v do."""

    @staticmethod
    def forward(ctx, x, v, kind, eps, keep, with_u, *prm):
        ctx.set_materialize_grads(False)
        x, v = _dense(x), _dense(v)
        prm = [None if p is None else p.contiguous() for p in prm]
        params = ops.NormParams(kind, eps, *prm)
        y = torch.empty_like(x)
        u = torch.empty_like(x) if with_u else None
        if keep == "8bit":
            kept = (ops.fno_norm_residual_saved_empty(x),)
            ops.fno_norm_residual_save(params, x, v, y, u, kept[0])
        else:
            kept = (x, v)
            ops.fno_norm_residual(params, x, v, y, u)
        ctx.kind, ctx.eps, ctx.n_kept = kind, eps, len(kept)
        ctx.save_for_backward(*kept, *prm)
        return y, u

    @staticmethod
    @once_differentiable
    def backward(ctx, gy, gu):
        none = (None,) * 6
        saved = ctx.saved_tensors
        kept, prm = saved[:ctx.n_kept], saved[ctx.n_kept:]
        need_x, need_v = ctx.needs_input_grad[:2]
        need = ctx.needs_input_grad[6:]
        if gy is None and gu is None or not (need_x or need_v or any(need)):
            return none + (None,) * len(prm)
        gu = _dense(gu)
        gy = torch.zeros_like(gu) if gy is None else _dense(gy)
        if gu is None:  # nothing came back through u: its norm's parameters have no gradient
            need = tuple(n and not name.endswith("_pre") for n, name in zip(need, ops._NORM_NAMES))
            if not (need_x or need_v or any(need)):
                return none + (None,) * len(prm)
        gx = torch.empty_like(gy) if need_x else None
        gv = torch.empty_like(gy) if need_v else None
        g = [torch.empty_like(p) if n else None for p, n in zip(prm, need)]
        ws = ops.fno_norm_residual_workspace_empty(gy) if any(need) else None
        params, grads = ops.NormParams(ctx.kind, ctx.eps, *prm), ops.NormGrads(*g)
        if ctx.n_kept == 1:
            ops.fno_norm_residual_backward_saved(params, kept[0], gy, gu, gx, gv, grads, ws)
        else:
            ops.fno_norm_residual_backward(params, kept[0], kept[1], gy, gu, gx, gv, grads, ws)
        return (gx, gv) + none[:4] + tuple(g)
