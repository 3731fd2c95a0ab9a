"""The binding's extension (csrc/binding.cpp) on tensors it cannot take."""

import sys

import torch

from spectral_convolution_amd import _training as ops


def test_tensors_without_storage_leave_nothing_behind():
    """A batched tensor inside vmap has no address: None, and nothing stays allocated of the attempt."""
    ops._t()
    kept = []

    def body(t):
        got = [ops._native.addresses(t, t, (4,)) for _ in range(2000)]
        before = sys.getallocatedblocks()
        for _ in range(2000):
            ops._native.addresses(t, t, (4,))
            ops._native.buffer(t, t, 8, 1)
        kept.append(sys.getallocatedblocks() - before)
        assert set(got) == {None}
        return t

    torch.vmap(body)(torch.zeros(3, 4))
    assert kept[0] < 500
