"""Sizes at the ends of what the training operators take, without a GPU: numbers that
do not fit the C ABI's integers are refused, not cut to their low bits."""

import pytest
import torch

import spectral_convolution_amd as fno

WIDE = 1 << 32


@pytest.mark.parametrize("call", [
    lambda: fno.fno_norm_residual_saved_bytes(WIDE + 1, 64, 1),
    lambda: fno.fno_norm_residual_saved_bytes(1, WIDE + 64, 1),
    lambda: fno.fno_norm_residual_workspace_bytes(WIDE + 1, 64, 1),
    lambda: fno.fno_channel_mix_saved_bytes(WIDE + 2, 4, 4, 10),
    lambda: fno.fno_channel_mix_saved_bytes(2, 4, 4, 10, act=WIDE + 1),
    lambda: fno.fno_channel_mix_workspace_bytes(2, 4, WIDE + 4, 10),
    lambda: fno.fno_channel_mix_workspace_bytes(2, 4, 4, (1 << 64) + 10),
    lambda: fno.fno_checkpoint_bytes((1 << 64) + 3, 32),
    lambda: fno.fno_checkpoint_bytes(3, (1 << 64) + 32),
])
def test_sizes_past_the_abis_integers(call):
    with pytest.raises(ValueError, match="range"):
        call()


def test_fields_past_the_abis_integers():
    """A batch of 2^32 + 1 tokens is not a batch of one (no memory behind these tensors)."""
    x = torch.empty(1, dtype=torch.float16).expand(WIDE + 1, 1)
    saved = torch.empty(512, dtype=torch.uint8)
    for call in (lambda: fno.fno_norm_residual(fno.NormParams("rms", 1e-5), x, x, x, None),
                 lambda: fno.fno_norm_residual_save(fno.NormParams("rms", 1e-5), x, x, x, None, saved),
                 lambda: fno.fno_norm_residual_backward(fno.NormParams("rms", 1e-5), x, x, x, None, x, None, None, None),
                 lambda: fno.fno_channel_mix_save(x, torch.empty(1, 1).half(), None, None, x, saved),
                 lambda: fno.fno_norm_residual_saved_empty(x), lambda: fno.fno_channel_mix_workspace_empty(x, 1)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()
