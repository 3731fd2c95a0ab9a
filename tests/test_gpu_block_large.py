"""The operators of a regularised block on fields whose offsets pass 32 bits: the last sample has what
it has in a call of its own."""

import pytest
import torch

import spectral_convolution_amd as fno

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
B, C, P = 3, 64, (1 << 31) // 192 * 2 + 1023  # 3 x 64 x P is past 2^32 values
TYPE = torch.float16


def field(seed, last):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty((B, P, C) if last else (B, C, P), dtype=TYPE, device=DEV)
    for b in range(B):
        x[b].normal_(generator=gen)
    return x


def close(got, want, tiny):
    """Within a step and a half of an fp16 result, or `tiny`."""
    for g, w in zip(got.flatten().split(1 << 28), want.flatten().split(1 << 28)):
        g, w = g.float(), w.float()
        assert bool(((g - w).abs() <= 3 * 2.0 ** -11 * torch.maximum(g.abs(), w.abs()) + tiny).all())


@pytest.mark.parametrize("last", (False, True), ids=("first", "last"))
def test_group_norm(last):
    assert B * C * P > 1 << 32
    x, gy = field(1, last), field(2, last)
    w = torch.linspace(0.5, 1.5, C, device=DEV).to(TYPE)
    p = fno.GroupNormParams(4, 1e-5, w, torch.zeros_like(w), 2, last)
    r = torch.empty(4, dtype=torch.float64, device=DEV)
    for i in range(4):
        own = (x[-1, :, 16 * i:16 * i + 16] if last else x[-1, 16 * i:16 * i + 16]).split(1 << 20 if last else 1)
        n = 16 * P
        mean = sum(c.double().sum() for c in own) / n
        r[i] = (sum(((c.double() - mean) ** 2).sum() for c in own) / n + 1e-5) ** -0.5
    out = []
    for a, g in ((x, gy), (x[-1:], gy[-1:])):
        y, gx, gw, gb = torch.empty_like(a), torch.empty_like(a), torch.empty_like(w), torch.empty_like(w)
        stats, ws = fno.fno_group_norm_stats_empty(a, 4), fno.fno_group_norm_workspace_empty(a, 4, last)
        fno.fno_group_norm(p, a, y, stats, ws)
        fno.fno_group_norm_backward(p, a, stats, g, gx, gw, gb, ws)
        out.append((y[-1], gx[-1]))
        # A lane's up to 2000 values wander by the root of their number of half steps, 45, which thousands of lanes average
        # to less than one; 40 joins by 7: a variance is off by 8 x 2^-24, and r by half of that and its own rounding.
        assert bool(((stats[-1, :, 1].double() - r) / r).abs().max() <= 6 * 2.0 ** -24)
        assert bool(torch.isfinite(gw).all()) and bool(torch.isfinite(gb).all())
    # The two calls cut a group into other pieces, so their statistics differ, by 12 x 2^-24 at most, and a result's
    # rounding by a step (two halves). Where gx = r (w gz - M1 - x^ M2) nearly vanishes that shows as it is: z moves by
    # 12 x 2^-24 z, so w gz by 1.5 (w) x 6.5 (the largest of 2^32 normal gy) x 0.3 (the largest |z act''(z)|) of
    # that, 35 x 2^-24; y, which vanishes with z (off by 2^-24 of a mean of 10^-4 beside that), by a subnormal's step.
    close(out[0][0], out[1][0], 3 * 2.0 ** -24)
    close(out[0][1], out[1][1], 36 * 2.0 ** -24)


def test_dropout_by_channels():
    v = field(3, True)
    y, alone = torch.empty_like(v), torch.empty_like(v)
    fno.fno_dropout_residual(fno.Dropout(0.5, 9, unit="channel"), None, v, y, True)
    kept = y[:, :7] != 0  # by the first pixels, whose values are 0 with a probability of 2^-13 or so each
    for b in range(B):
        torch.mul(v[b], kept[b].any(0).to(TYPE) * 2, out=alone[b])
        assert torch.equal(y[b], alone[b])
    assert 0 < int(kept.any(1).sum()) < B * C


def test_kept_in_four_bits_and_mixed():
    x = field(4, False)
    weight = torch.randn(16, C, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5)).to(TYPE)
    whole, alone = fno.fno_mx4_empty(x), fno.fno_mx4_empty(x[-1:])
    fno.fno_mx4_pack(x, whole)
    fno.fno_mx4_pack(x[-1:], alone)
    back, own = torch.empty_like(x), torch.empty_like(x[-1:])
    fno.fno_mx4_unpack(whole, back)
    fno.fno_mx4_unpack(alone, own)
    assert torch.equal(back[-1], own[0])
    del back, own
    A = fno.Mx4Weight(weight)
    y, ya = (torch.empty((n, 16, P), dtype=TYPE, device=DEV) for n in (B, 1))
    fno.fno_channel_mix_mx4(whole, A.packed, None, None, y, C, 1)
    fno.fno_channel_mix_mx4(alone, A.packed, None, None, ya, C, 1)
    assert torch.equal(y[-1], ya[0])
