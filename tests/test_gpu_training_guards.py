"""Nothing is written outside the outputs: each lies between guard bytes that have to stay
as they were, at shapes that end inside a tile, a block or a 16-byte access; inputs stay too."""

import pytest
import torch

import spectral_convolution_amd as fno
from training_util import DT, NORM_NAMES

pytestmark = pytest.mark.gpu
DTYPES = ["f32", "f16", "bf16"]
GUARD = 4096


class Arena:
    """Device memory of a known pattern, tensors carved out of it at 256-byte boundaries."""

    def __init__(self, room):
        self.mem = torch.full((room,), 0xA5, dtype=torch.uint8, device="cuda")
        self.at, self.held = GUARD, []

    def take(self, shape, dtype):
        n = int(torch.Size(shape).numel()) * torch.empty(0, dtype=dtype).element_size()
        t = self.mem[self.at:self.at + n].view(dtype).view(shape)
        assert t.data_ptr() % 256 == 0
        self.held.append((self.at, n))
        self.at += -(-(n + GUARD) // 256) * 256
        assert self.at + GUARD < self.mem.numel()
        return t

    def check(self):
        keep = torch.ones(self.mem.numel(), dtype=torch.bool, device="cuda")
        for a, n in self.held:
            keep[a:a + n] = False
        hit = torch.nonzero(keep & (self.mem != 0xA5))
        assert hit.numel() == 0, f"byte {int(hit[0])} of the guards was written, outputs at {self.held}"


def _inputs(dtype, *shapes):
    gen = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(s, generator=gen, device="cuda").to(DT[dtype]) for s in shapes]


def _unchanged(pairs):
    for t, before in pairs:
        assert torch.equal(t.view(torch.uint8) if t.dtype != torch.uint8 else t, before)


def _bytes(ts):
    return [(t, (t.view(torch.uint8) if t.dtype != torch.uint8 else t).clone()) for t in ts]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("shape", [(1, 1, 2), (3, 7, 33), (2, 13, 63), (2, 20, 95), (530, 17, 3), (520, 60, 7), (515, 100, 9),
                                   (2, 130, 127), (1, 257, 31), (2, 511, 65), (1, 1), (5, 3), (2, 63), (9, 257), (1030, 41),
                                   (3, 1001), (2, 3001), (1, 8191)], ids=str)
def test_norm(dtype, kind, shape):
    B, C = shape[:2]
    x, v, gy, gu = _inputs(dtype, *[shape] * 4)
    p = dict(zip(NORM_NAMES, _inputs(dtype, *[(B, C) if k == "gate" else (C,) for k in NORM_NAMES])))
    N = fno.NormParams(kind, 1e-5, **p)
    kept, work = fno.fno_norm_residual_saved_empty(x).numel(), fno.fno_norm_residual_workspace_empty(x).numel()
    a = Arena(8 * x.numel() * x.element_size() + kept + work + 4 * B * C * 4 + 32 * (GUARD + 512) + 64 * C)
    y, u, gx, gv, fx, fv = (a.take(shape, DT[dtype]) for _ in range(6))
    saved, ws = a.take((kept,), torch.uint8), a.take((work,), torch.uint8)
    G = fno.NormGrads(**{k: a.take(tuple(t.shape), DT[dtype]) for k, t in p.items()})
    before = _bytes([x, v, gy, gu, *p.values()])
    fno.fno_norm_residual(N, x, v, y, u)
    fno.fno_norm_residual_save(N, x, v, y, u, saved)
    fno.fno_norm_residual_backward_saved(N, saved, gy, gu, gx, gv, G, ws)
    fno.fno_norm_residual_backward(N, x, v, gy, gu, fx, fv, G, ws)
    a.check()
    _unchanged(before)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("B,I,O,P", [(1, 1, 1, 1), (3, 5, 7, 33), (2, 17, 16, 63), (2, 16, 17, 65), (2, 33, 31, 127), (1, 65, 64, 129),
                                     (2, 64, 65, 31), (1, 127, 128, 95), (2, 128, 3, 257), (2, 3, 127, 255), (2300, 9, 20, 5)])
@pytest.mark.parametrize("act,add", [(1, True), (0, True), (1, False)])
def test_mix(dtype, B, I, O, P, act, add):
    x, A, bias, ad, gy = _inputs(dtype, (B, I, P), (O, I), (O,), (B, O, P), (B, O, P))
    ad = ad if add else None
    kept, work = fno.fno_channel_mix_saved_empty(x, O, act, add).numel(), fno.fno_channel_mix_workspace_empty(x, O).numel()
    a = Arena(2 * (x.numel() + 3 * gy.numel() + A.numel()) * 4 + kept + work + 16 * (GUARD + 512))
    y, gx, gA, gb = (a.take(s, DT[dtype]) for s in ((B, O, P), (B, I, P), (O, I), (O,)))
    gadd = a.take((B, O, P), DT[dtype]) if add else None
    saved, ws = a.take((kept,), torch.uint8), a.take((work,), torch.uint8)
    before = _bytes([t for t in (x, A, bias, ad, gy) if t is not None])
    fno.fno_channel_mix_save(x, A, bias, ad, y, saved, act)
    fno.fno_channel_mix_backward_saved(saved, A, bias, gy, gx, gA, gb, gadd, ws, act, add)
    a.check()
    _unchanged(before)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (7, 3), (3, 31), (5, 33), (2, 257), (96, 3721), (1, 100003)])
def test_checkpoint(dtype, rows, n):
    (x,) = _inputs(dtype, (rows, n))
    kept = fno.fno_checkpoint_bytes(rows, n)
    a = Arena(kept + x.numel() * 4 + 4 * (GUARD + 512))
    saved, y = a.take((kept,), torch.uint8), a.take((rows, n), DT[dtype])
    before = _bytes([x])
    fno.fno_checkpoint_pack(x, saved)
    fno.fno_checkpoint_unpack(saved, y)
    a.check()
    _unchanged(before)
