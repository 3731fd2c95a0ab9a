"""Group norm where a lane's sums are longest and where its launches are largest."""

import pytest
import torch

import spectral_convolution_amd as fno

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("groups", (32, 1), ids=("runs", "pieces"))
def test_gradients_of_parameters_over_long_runs(groups):
    """2^20 equal terms 1 + 2^-15 in fp32: from 512 on a sum that takes one after the other loses the small part of each, always
    to the same side. Stretches of 256 are exact, and so is everything joined from them."""
    C, rows = 1024, 1 << 20
    shape = (rows, C) if groups > 1 else (1, rows, C)
    x = torch.ones(shape, device=DEV)
    gy = torch.full(shape, 1 + 2.0 ** -15, device=DEV)
    stats = fno.fno_group_norm_stats_empty(x, groups)
    stats[..., 0], stats[..., 1] = 0.0, 1.0  # x^ = x
    w, b = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    gw, gb = torch.empty_like(w), torch.empty_like(b)
    prm = fno.GroupNormParams(groups, 1e-5, w, b, channels_last=True)
    ws = fno.fno_group_norm_workspace_empty(x, groups, True)
    fno.fno_group_norm_backward(prm, x, stats, gy, None, gw, gb, ws)
    want = rows + rows * 2.0 ** -15
    assert (gb == want).all() and (gw == want).all()


def test_variance_of_long_pieces():
    """Squares (1 + 2^-8)^2 = 1 + 2^-7 + 2^-16 lose their last digit in sums past 256, always to the same side.
    Values: 0, -s, s, -s, ... in every 256 rows: their sum is -s, that of their squares 255 s^2."""
    C, P, G, eps = 2048, 1 << 20, 8, 1e-5
    s = 1 + 2.0 ** -8
    row = torch.full((256,), s, device=DEV)
    row[1::2] = -s
    row[0] = 0
    x = torch.empty((1, P, C), dtype=torch.float16, device=DEV)
    x.view(P // 256, 256, C)[:] = row.half()[None, :, None]
    y = torch.empty_like(x)
    stats = fno.fno_group_norm_stats_empty(x, G)
    fno.fno_group_norm(fno.GroupNormParams(G, eps, channels_last=True), x, y, stats,
                       fno.fno_group_norm_workspace_empty(x, G, True))
    mean, var = -s / 256, s * s * (255 / 256 - 2.0 ** -16)
    st = stats.double()
    assert ((st[..., 0] - mean).abs() <= 8 * 2.0 ** -24 * s).all()
    # half steps of r: one of each stretch's variance, of the division, of eps added and of the result, two of the root
    assert ((st[..., 1] * (var + eps) ** 0.5 - 1).abs() <= 6 * 2.0 ** -24).all()


def test_millions_of_groups_of_1024_threads():
    """2^22 groups that 1024 threads hold each: fewer workgroups than groups, equal to a call on some of them."""
    n, P, G = 1024, 8200, 1 << 22
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of GPU memory")
    prm = fno.GroupNormParams(1, 1e-5, act=2)
    gen = torch.Generator(device=DEV).manual_seed(1)
    part = torch.randn((n, 1, P), generator=gen, device=DEV).half()
    ws = fno.fno_group_norm_workspace_empty(part, 1)
    y, stats, gx = torch.empty_like(part), fno.fno_group_norm_stats_empty(part, 1), torch.empty_like(part)
    fno.fno_group_norm(prm, part, y, stats, ws)
    fno.fno_group_norm_backward(prm, part, stats, part, gx, None, None, ws)
    x = torch.empty((G, 1, P), dtype=torch.float16, device=DEV)
    x.view(G // n, n, 1, P)[:] = part
    out, stats_all = torch.full_like(x, 7.0), fno.fno_group_norm_stats_empty(x, 1)
    ws = fno.fno_group_norm_workspace_empty(x, 1)
    fno.fno_group_norm(prm, x, out, stats_all, ws)
    assert (stats_all.view(G // n, *stats.shape) == stats).all()
    for o in out.view(G // n, n, 1, P).split(256):
        assert (o == y).all()
    fno.fno_group_norm_backward(prm, x, stats_all, x, out, None, None, ws)
    for o in out.view(G // n, n, 1, P).split(256):
        assert (o == gx).all()
