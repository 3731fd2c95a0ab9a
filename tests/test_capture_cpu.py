"""The check of a captured backward's leaves (spectral_convolution_amd/_capture.py), on the CPU with a capture pretended."""

from types import SimpleNamespace

import pytest
import torch

from spectral_convolution_amd import _capture, _training

GPU = SimpleNamespace(is_cuda=True)


class Pass(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, b, c):
        return a + b + c

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gy):
        _capture.check_backward(ctx, GPU)
        return gy, gy, gy


ELSEWHERE = ((0, 0, 1),)  # the default stream


def _backward(monkeypatch, capturing, elsewhere):
    seen = []
    _training._t()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(_training, "_native", SimpleNamespace(elsewhere=lambda *t: seen.extend(t) or list(elsewhere)))
    a, b = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    got = torch.autograd.grad(Pass.apply(a, 2 * b, torch.ones(3)).sum(), (a, b))
    assert all((g == k).all() for g, k in zip(got, (1, 2)))
    return seen, a


def test_leaves_are_looked_at_in_a_capture(monkeypatch):
    seen, a = _backward(monkeypatch, True, ())
    assert len(seen) == 1 and seen[0] is a  # not what was computed from b, not the constant
    assert _backward(monkeypatch, False, ELSEWHERE)[0] == []


def test_leaves_elsewhere_are_refused(monkeypatch):
    with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
        _backward(monkeypatch, True, ELSEWHERE)


def test_streams_of_the_capture_are_no_reason(monkeypatch):
    """A stream that has joined the capture is part of it; one that has not is refused, among others too."""
    monkeypatch.setattr(_capture, "_captured", lambda stream_id, *_: stream_id == 5)
    _backward(monkeypatch, True, ((5, 0, 1),))
    with pytest.raises(RuntimeError, match="belongs to an autograd graph"):
        _backward(monkeypatch, True, ((5, 0, 1), (6, 0, 1)))


def test_leaves_of_the_current_stream():
    _training._t()
    a = torch.ones(2, requires_grad=True)
    kept = a * 2
    assert _training._native.elsewhere(a, None, kept) == []


def test_no_gradient(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    _capture.check_backward(None, None)
    _capture.check_backward(None, torch.ones(1))


def test_every_function_checks_its_backward():
    """Each autograd Function of the framework begins its backward with the check."""
    import inspect

    import spectral_convolution_amd as fno
    from spectral_convolution_amd import _block_autograd as block, _training_autograd as training
    for f in (block.GroupNormFunction, block.DropoutResidualFunction, training.ChannelMixFunction, training.NormResidualFunction,
              fno.SpectralConvFunction):
        source = inspect.getsource(inspect.unwrap(f.backward))
        assert source.index("check_backward(ctx, g") < source.index("torch.empty_like"), f.__name__
