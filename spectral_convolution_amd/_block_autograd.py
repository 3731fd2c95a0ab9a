"""The operators of a regularised block as PyTorch autograd Functions: group norm
with an activation and dropout, and dropout into a residual stream. Imported on first
use, since it imports torch. Every value is computed in the library's kernels;
torch allocates the tensors."""

import torch
from torch.autograd.function import once_differentiable

from . import _block_ops as ops
from ._capture import check_backward
from ._training_autograd import _dense


class GroupNormFunction(torch.autograd.Function):
    """y = D(act(group norm of x))."""

    @staticmethod
    def forward(ctx, x, weight, bias, params, dropout):
        x = _dense(x)
        weight = None if weight is None else weight.contiguous()
        bias = None if bias is None else bias.contiguous()
        p = ops.GroupNormParams(params.groups, params.eps, weight, bias, params.act, params.channels_last)
        y = torch.empty_like(x)
        stats = ops.fno_group_norm_stats_empty(x, p.groups) if any(ctx.needs_input_grad) else None
        ws = ops.fno_group_norm_workspace_empty(x, p.groups, p.channels_last)
        ops.fno_group_norm(p, x, y, stats, ws, dropout)
        ctx.spec, ctx.dropout = (p.groups, p.eps, p.act, p.channels_last), dropout
        ctx.save_for_backward(x, weight, bias, stats)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        check_backward(ctx, gy)
        x, weight, bias, stats = ctx.saved_tensors
        need = ctx.needs_input_grad
        groups, eps, act, last = ctx.spec
        gy = _dense(gy)
        gx = torch.empty_like(x) if need[0] else None
        gw = torch.empty_like(weight) if need[1] else None
        gb = torch.empty_like(bias) if need[2] else None
        if gx is None and gw is None and gb is None:
            return (None,) * 5
        p = ops.GroupNormParams(groups, eps, weight, bias, act, last)
        ws = ops.fno_group_norm_workspace_empty(x, groups, last)
        ops.fno_group_norm_backward(p, x, stats, gy, gx, gw, gb, ws, ctx.dropout)
        return gx, gw, gb, None, None


class DropoutResidualFunction(torch.autograd.Function):
    """y = x + D(v)."""

    @staticmethod
    def forward(ctx, v, x, dropout, channels_last):
        v, x = _dense(v), _dense(x)
        y = torch.empty_like(v)
        ops.fno_dropout_residual(dropout, x, v, y, channels_last)
        ctx.dropout, ctx.last = dropout, channels_last
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, gy):
        check_backward(ctx, gy)
        gv = None
        if ctx.needs_input_grad[0]:
            g = _dense(gy)
            gv = torch.empty_like(g)
            ops.fno_dropout_residual(ctx.dropout, None, g, gv, ctx.last)
        return gv, gy if ctx.needs_input_grad[1] else None, None, None
