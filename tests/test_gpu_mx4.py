"""GPU parity of the 4-bit floats: codes and scales have to be equal to their definition's
(oracle/block.py), the channel mix of packed operands within its roundings."""

import numpy as np
import pytest
import torch

import spectral_convolution_amd as fno
from oracle import block as ref
from training_util import CHAIN, DT, close, f64, stored

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DTYPES = ["f32", "f16", "bf16"]


def parts(packed, rows, C):
    nb = -(-C // 32)
    b = packed.cpu().numpy()
    q = b[:rows * nb * 16].reshape(rows, nb, 16)
    at = -(-rows * nb * 16 // 256) * 256
    return np.stack([q & 15, q >> 4], -1).reshape(rows, nb, 32), b[at:at + rows * nb].reshape(rows, nb)


def pack(x):
    packed = torch.full((fno.fno_mx4_bytes(x.shape[0], x.shape[1], x[0, 0].numel()),), 77, dtype=torch.uint8, device=DEV)
    fno.fno_mx4_pack(x.to(DEV), packed)
    return packed


def check_kept(x, x64):
    """Codes, scales and the values read back are the definition's."""
    packed = pack(x)
    rows = ref.mx4_rows(x64)
    q, s = ref.mx4(rows)
    gq, gs = parts(packed, len(rows), rows.shape[1])
    assert (gs == s).all() and (gq == q).all()
    y = torch.full_like(x.to(DEV), 3.0)
    fno.fno_mx4_unpack(packed, y)
    assert np.array_equal(f64(y), ref.mx4_trip(x64), equal_nan=True)
    return packed


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (3, 31), (2, 32), (5, 33), (300, 40), (7, 1000), (2, 8192), (1, 65536), (1, 1, 2),
                                   (2, 4, 256), (3, 33, 7), (1, 64, 1001), (2, 130, 3), (5, 7, 5), (2, 96, 65), (70, 40, 33)],
                         ids=str)
def test_kept_values(dtype, shape):
    x, x64 = stored(np.random.default_rng(sum(shape)), shape, dtype, spread=True)
    check_kept(x, x64)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("field", [False, True])
def test_ties_and_ends(dtype, field):
    """Every border between codes, from both sides, at scales from the type's lowest to its highest."""
    fi = torch.finfo(DT[dtype])
    least = {"f32": -149, "f16": -24, "bf16": -133}[dtype]
    most = int(np.log2(fi.max))
    rows = []
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.5])
    near = np.concatenate([borders, borders * (1 + float(fi.eps)), borders * (1 - float(fi.eps))])
    for e in (least, least + 1, least + 3, -126, -127, -125, -14, 0, 5, most - 2):
        if e < least:
            continue
        rows.append(np.concatenate([near, [4.0, -0.0]]) * 2.0 ** e)
        rows.append(-np.concatenate([near[:15], [7.9375] * 17]) * 2.0 ** e)
    rows += [np.zeros(32), -np.zeros(32), np.full(32, float(fi.max)), np.full(32, 2.0 ** least), np.full(32, float(fi.tiny))]
    x = torch.tensor(np.array(rows)).to(DT[dtype])
    if field:
        x = x.t().reshape(1, 32, -1).contiguous()
    check_kept(x, x.double().numpy())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("field", [False, True])
def test_poisoned_blocks(dtype, field):
    x = torch.ones(5, 100)
    x[0, 5], x[1, 40], x[2, 99], x[3, 63] = float("nan"), float("inf"), -float("inf"), -float("nan")
    x = x.to(DT[dtype])
    if field:
        x = x.t().reshape(1, 100, 5).contiguous()
    check_kept(x, x.double().numpy())


# ------------------------------------------------------------------ products

def mix(dtype, B, I, O, P, act, add, bias, seed=0, poison=None):
    rng = np.random.default_rng(seed)
    shape = (B, I) if P == 1 else (B, I, P)
    x, x64 = stored(rng, shape, dtype, spread=True)
    A, A64 = stored(rng, (O, I), dtype, I ** -0.5)
    b, b64 = stored(rng, (O,), dtype, 0.3) if bias else (None, None)
    out = (B, O) if P == 1 else (B, O, P)
    d, d64 = stored(rng, out, dtype) if add else (None, None)
    y = torch.full(out, 7.0, dtype=DT[dtype], device=DEV)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    fno.fno_channel_mix_mx4(pack(x), pack(A), dev(b), dev(d), y, I, act=act)
    x3 = ref.mx4_trip(x64).reshape(B, I, P)
    want, size = ref.mx4_mix(x3, ref.mx4_trip(A64), b64, None if d64 is None else d64.reshape(B, O, P), act)
    return y, want.reshape(out), size.reshape(out)


# (B, I, O, P): one value, block and step ends, tile ends in rows and columns, tokens and fields, few and many rows
MIXES = [(1, 1, 1, 1), (1, 33, 5, 1), (2, 128, 64, 1), (17, 129, 70, 1), (300, 200, 257, 1), (1, 4096, 96, 1), (3, 1000, 33, 1),
         (16, 512, 512, 1), (33, 512, 130, 1), (260, 544, 513, 1), (1, 32, 1, 2), (2, 4, 4, 256), (3, 31, 7, 5), (2, 64, 64, 300),
         (1, 200, 72, 1001), (4, 96, 130, 17), (5, 40, 3, 63), (1, 512, 300, 515)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", MIXES, ids=str)
def test_mix(dtype, shape):
    i = MIXES.index(shape)
    for act, add, bias in ((0, False, False), (1, True, True), (i % 2, i % 3 == 0, True)):
        y, want, size = mix(dtype, *shape, act, add, bias, seed=i)
        close("y", y, want, dtype, size=size)


def random_packed(gen, rows, C):
    """(packed, values in float64 [rows][C]): any codes, scales around 1."""
    nb = -(-C // 32)
    code = torch.randint(0, 16, (rows, nb, 32), generator=gen, device=DEV, dtype=torch.uint8)
    code.view(rows, -1)[:, C:] = 0
    scale = torch.randint(120, 135, (rows, nb), generator=gen, device=DEV, dtype=torch.uint8)
    at = -(-rows * nb * 16 // 256) * 256
    packed = torch.zeros(fno.fno_mx4_bytes(rows, C), dtype=torch.uint8, device=DEV)
    packed[:rows * nb * 16] = (code[..., ::2] | code[..., 1::2] << 4).view(-1)
    packed[at:at + rows * nb] = scale.view(-1)
    v = torch.from_numpy(np.concatenate([ref.MX4_VALUES, -ref.MX4_VALUES])).to(DEV)[code.long()]
    v = v * torch.exp2(scale.double() - 127)[..., None]
    return packed, v.view(rows, -1)[:, :C]


# rows of either operand and the sum's length: tiles of 128 and 256 whole and cut, sums that end in the
# first and second half of a stage of 256, one to many stages, and the kernels beside
LARGE = [(65, 128, 512), (128, 256, 640), (129, 127, 768), (300, 200, 896), (257, 700, 1024),
         (96, 1000, 1152), (400, 300, 4096), (3000, 3100, 512), (2900, 3300, 1920), (4096, 2304, 640),
         (130, 140, 500), (300, 300, 600), (70, 66, 992), (64, 4096, 4096), (40, 3000, 1100), (3, 500, 1100),
         (20, 300, 1024), (20, 300, 1100), (3600, 3500, 640), (3500, 3600, 1408), (2100, 2100, 100)]


@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_large_products(shape):
    B, O, I = shape
    gen = torch.Generator(device=DEV).manual_seed(B)
    (xq, x), (aq, a) = random_packed(gen, B, I), random_packed(gen, O, I)
    z, size = x @ a.t(), x.abs() @ a.t().abs()
    for dtype, act in (("f32", 0), ("bf16", 1), ("f16", 0)):
        bias = torch.randn(O, generator=gen, device=DEV).to(DT[dtype])
        add = torch.randn(B, O, generator=gen, device=DEV).to(DT[dtype]) if act == 0 else None
        scale = 2.0 ** -9 if dtype == "f16" else 1.0  # sums of up to some thousands stay in range
        y = torch.full((B, O), float("nan"), dtype=DT[dtype], device=DEV)
        q = xq.clone()
        if dtype == "f16":
            at = -(-B * -(-I // 32) * 16 // 256) * 256
            q[at:at + B * -(-I // 32)] -= 9
        fno.fno_channel_mix_mx4(q, aq, bias, add, y, I, act=act)
        want = z * scale + bias.double() + (0 if add is None else add.double())
        terms = size * scale + bias.double().abs() + (0 if add is None else add.double().abs())
        want = want * torch.special.ndtr(want) if act else want
        bound = float(torch.finfo(DT[dtype]).eps) / 2 * want.abs() * 1.001 + CHAIN * terms + 2.0 ** -25
        assert ((y.double() - want).abs() <= bound).all(), (dtype, act)


@pytest.mark.parametrize("shape", [(2, 512, 100, 300), (3, 640, 300, 129), (1, 1024, 70, 1000), (9, 512, 513, 700)], ids=str)
def test_large_products_of_fields(shape):
    B, I, O, P = shape
    gen = torch.Generator(device=DEV).manual_seed(P)
    (xq, x), (aq, a) = random_packed(gen, B * P, I), random_packed(gen, O, I)
    fold = lambda t: t.view(B, P, O).transpose(1, 2)  # noqa: E731
    bias = torch.randn(O, generator=gen, device=DEV)
    add = torch.randn(B, O, P, generator=gen, device=DEV)
    y = torch.full((B, O, P), float("nan"), device=DEV)
    fno.fno_channel_mix_mx4(xq, aq, bias, add, y, I)
    want = fold(x @ a.t()) + bias.double().view(1, O, 1) + add.double()
    terms = fold(x.abs() @ a.t().abs()) + bias.double().abs().view(1, O, 1) + add.double().abs()
    assert ((y.double() - want).abs() <= 2.0 ** -24 * want.abs() + CHAIN * terms).all()


def test_poisoned_block_poisons_its_products():
    for P in (1, 40):
        x = torch.ones((4, 100) if P == 1 else (4, 100, P), device=DEV)
        A = torch.ones(20, 100, device=DEV)
        x[2, 50] = float("nan")
        A[7, 99] = float("inf")
        y = torch.empty((4, 20) if P == 1 else (4, 20, P), device=DEV)
        fno.fno_channel_mix_mx4(pack(x), pack(A), None, None, y, 100)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[2], bad[:, 7] = True, True
        assert torch.isnan(y[bad]).all() and (y[~bad] == 100).all()


def test_wide_scales():
    """Operands whose scales lie at opposite ends multiply to ordinary values."""
    x, A = torch.randn(40, 256, device=DEV), torch.randn(30, 256, device=DEV)
    y, big = torch.empty(40, 30, device=DEV), torch.empty(40, 30, device=DEV)
    fno.fno_channel_mix_mx4(pack(x), pack(A), None, None, y, 256)
    fno.fno_channel_mix_mx4(pack(x * 2.0 ** 110), pack(A * 2.0 ** -110), None, None, big, 256)
    assert torch.equal(y, big)


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    for shape in ((1, 2048, 300), (200, 600, 300)):
        B, I, O = shape
        x, A = torch.randn(B, I, device=DEV), torch.randn(O, I, device=DEV)
        xq, Aq = fno.fno_mx4_empty(x), pack(A)
        y, want = torch.empty(B, O, device=DEV), torch.empty(B, O, device=DEV)

        def step(out):
            fno.fno_mx4_pack(x, xq)
            fno.fno_channel_mix_mx4(xq, Aq, None, None, out, I, act=1)

        step(want)
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.Stream()):
            step(y)
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(y)
        for _ in range(3):
            y.zero_()
            x.mul_(1.5)
            step(want)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 40, 21, 1), (2, 40, 21, 35), (1, 600, 513, 1), (300, 512, 260, 1)], ids=str)
def test_guards(dtype, shape):
    """Nothing is written beside the outputs."""
    B, I, O, P = shape
    x = torch.randn((B, I) if P == 1 else (B, I, P), device=DEV).to(DT[dtype])
    A = torch.randn(O, I, device=DEV)
    size = fno.fno_mx4_bytes(B, I, P)
    buf = torch.full((size + 512,), 99, dtype=torch.uint8, device=DEV)
    fno.fno_mx4_pack(x, buf[256:256 + size])
    assert (buf[:256] == 99).all() and (buf[256 + size:] == 99).all()
    n = B * O * P
    out = torch.full((n + 128,), 3.0, dtype=DT[dtype], device=DEV)
    y = out[64:64 + n].view((B, O) if P == 1 else (B, O, P)).fill_(float("nan"))
    fno.fno_channel_mix_mx4(buf[256:256 + size], pack(A), None, None, y, I)
    assert (out[:64] == 3).all() and (out[64 + n:] == 3).all() and torch.isfinite(y).all()
    n = x.numel()
    out = torch.full((n + 128,), 3.0, dtype=DT[dtype], device=DEV)
    fno.fno_mx4_unpack(buf[256:256 + size], out[64:64 + n].view(x.shape))
    assert (out[:64] == 3).all() and (out[64 + n:] == 3).all()


@pytest.mark.parametrize("grid", [(), (5, 7), (3, 4, 5)], ids=str)
def test_serving_call(grid):
    x = torch.randn(2, 70, *grid, device=DEV)
    A, b, add = torch.randn(33, 70, device=DEV), torch.randn(33, device=DEV), torch.randn(2, 33, *grid, device=DEV)
    w = fno.Mx4Weight(A)
    y = fno.channel_mix_mx4(x, w, b, add, act=1)
    P = x[0, 0].numel()
    x3 = ref.mx4_trip(f64(x).reshape(2, 70, P))
    want, size = ref.mx4_mix(x3, ref.mx4_trip(f64(A)), f64(b), f64(add).reshape(2, 33, P), 1)
    close("y", y.reshape(2, 33, P), want, "f32", size=size)
    strided = torch.randn(70, 2, *grid, device=DEV).transpose(0, 1)
    assert torch.equal(fno.channel_mix_mx4(strided, w), fno.channel_mix_mx4(strided.contiguous(), w))
    with pytest.raises(ValueError, match="gradient"):
        fno.channel_mix_mx4(x.requires_grad_(), w)
    with torch.no_grad():
        assert torch.equal(fno.channel_mix_mx4(x, w, b, add, act=1), y)
    with pytest.raises(ValueError, match="channels"):
        fno.channel_mix_mx4(x.detach()[:, :69].contiguous(), w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 40, 1024), (2, 70, 4096), (5, 96, 1020), (1, 33, 2052), (40, 64, 52), (2, 200, 514)], ids=str)
def test_kept_values_of_whole_workgroups(dtype, shape):
    """Pixels of a workgroup that follow each other over samples' ends, odd and even numbers of blocks."""
    B, C, P = shape
    gen = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn(shape, generator=gen, device=DEV).mul_(torch.exp2(torch.randint(-4, 5, (B, C, 1), generator=gen, device=DEV)))
    x = x.to(DT[dtype])
    packed = pack(x)
    rows = x.transpose(1, 2).reshape(B * P, C).contiguous()  # tokens, whose codes the other tests hold to the definition
    want = pack(rows)
    nb = -(-C // 32)
    at = -(-B * P * nb * 16 // 256) * 256
    assert torch.equal(packed[:B * P * nb * 16], want[:B * P * nb * 16])
    assert torch.equal(packed[at:at + B * P * nb], want[at:at + B * P * nb])
