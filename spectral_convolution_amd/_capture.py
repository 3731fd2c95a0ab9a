"""Captured graphs and autograd. A leaf's gradient accumulator belongs to the stream that was current when the first
autograd graph holding the leaf was made, and lives as long as something keeps it: that graph (its outputs), a hook on it.
A backward that is captured on another stream would wait for that one, and unless it has joined the capture the end of the capture would
end the process; these checks raise an error before."""

import torch

from . import _training as ops


def _captured(stream_id, device_index, device_type):
    """Whether a stream has joined a capture. The default stream cannot, and is not asked."""
    if stream_id == 0:
        return False
    with torch.cuda.stream(torch.cuda.Stream(stream_id=stream_id, device_index=device_index, device_type=device_type)):
        return torch.cuda.is_current_stream_capturing()


def _check(leaves):
    ops._t()
    if all(_captured(*s) for s in ops._native.elsewhere(*leaves)):
        return
    raise RuntimeError("a leaf of this call belongs to an autograd graph that lives on another stream: drop "
                       "that graph (its outputs, and hooks on the leaf's gradient accumulator) before capturing a backward of "
                       "the same leaves, or run it on the stream that captures")


def check_call(*inputs):
    """Refuse a captured call of leaves that belong elsewhere, at the call. A captured forward whose
    backward is not wanted runs under torch.no_grad()."""
    if inputs[0].is_cuda and torch.is_grad_enabled() and torch.cuda.is_current_stream_capturing():
        _check(inputs)


def check_backward(ctx, grad):
    """Refuse, from inside a captured backward, to pass gradients on to leaves that belong elsewhere."""
    if grad is not None and grad.is_cuda and torch.cuda.is_current_stream_capturing():
        _check([node.variable for node, _ in ctx.next_functions if hasattr(node, "variable")])
