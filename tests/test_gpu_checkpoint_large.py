"""Checkpoints past 2^32 units of 8 values: the grid's second dimension and offsets beyond 32 bits."""

import pytest
import torch

import spectral_convolution_amd as fno

pytestmark = pytest.mark.gpu


def test_checkpoint_of_a_billion_short_rows():
    """2^30 + 5000 rows of one value: 33 bytes a row, 35 GB in all. Whole numbers of 7 bits are kept exactly."""
    rows = (1 << 30) + 5000
    need = fno.fno_checkpoint_bytes(rows, 1) + 4 * rows
    if torch.cuda.mem_get_info()[0] < 1.2 * need:
        pytest.skip("needs 40 GB of device memory")
    x = torch.randint(-127, 128, (rows, 1), dtype=torch.int8, device="cuda").half()
    saved = torch.empty(fno.fno_checkpoint_bytes(rows, 1), dtype=torch.uint8, device="cuda")
    y = torch.full_like(x, 7.0)
    fno.fno_checkpoint_pack(x, saved)
    fno.fno_checkpoint_unpack(saved, y)
    assert torch.equal(x, y)
    # the last rows' codes and exponents by hand: 64 <= |q| < 128, x = q 2^e
    tail = saved[32 * (rows - 100):32 * rows].view(torch.int8).view(100, 32)
    off = (32 * rows + 255) // 256 * 256
    e = saved[off + rows - 100:off + rows].view(torch.int8).double()
    want = x[-100:, 0].double()
    assert torch.equal(tail[:, 0].double() * torch.exp2(e) * (want != 0), want) and (tail[:, 1:] == 0).all()
