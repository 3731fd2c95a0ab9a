"""Cases of the operators of a regularised block and of its 4-bit serving form:
group norm with an activation and dropout, dropout into a residual stream, and
microscaled 4-bit floats with the channel mix of two operands kept in them.

Fields are [batch][channels][pixels], channels-last ones [batch][pixels][channels].
With `own` true run() calls the library; otherwise it computes the same outputs
with elementary torch operations in fp32 (fp64 for sums over a group), rounded
once at the end. exact() computes them in fp64 from the definitions, gradients by
automatic differentiation, random bits by arithmetic on 16-bit halves.

Operators ("op" of a case):
  gn_fwd    y = drop(act(group norm of x))
  gn_step   that forward, then its backward: gradients of x, weight and bias
  drop      y = x + drop(v), or drop(v) alone (also the backward of both)
  mx4_keep  a field or tokens to 4-bit floats and back
  mx4_mix   y = act(A x + bias + add), A and x in 4-bit floats already
  mx4_serve the same on x in its storage type, packed within the call
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5
_BLOCK = 32        # values that share one power of two in the 4-bit format
_LOW32 = 0xFFFFFFFF


# ------------------------------------------------------------------- cases

def listed():
    return [
        # training of the network configuration with group norm, 8 channels a group: the largest norm
        dict(name="gn_step 20x64x256^2 f16", op="gn_step", batch=20, channels=64, pixels=65536, groups=8, act=1,
             last=False, p=0.0, unit="element", dtype="f16"),
        # the smallest layer configuration: a call's latency
        dict(name="gn_fwd 2x4x16^2 f32", op="gn_fwd", batch=2, channels=4, pixels=256, groups=2, act=0, last=False,
             p=0.0, unit="element", dtype="f32"),
        # channels last, as data sets and point-wise networks hold fields
        dict(name="gn_fwd 16x128^2x128 last bf16", op="gn_fwd", batch=16, channels=128, pixels=16384, groups=32,
             act=2, last=True, p=0.0, unit="element", dtype="bf16"),
        # the 64^3 configuration, fp32, channels last, dropout behind the activation
        dict(name="gn_step 4x64^3x32 last f32", op="gn_step", batch=4, channels=32, pixels=262144, groups=4, act=1,
             last=True, p=0.1, unit="element", dtype="f32"),
        # ragged: 61 x 61 grid, groups of 16 channels, dropout
        dict(name="gn_step 3x48x61^2 bf16", op="gn_step", batch=3, channels=48, pixels=3721, groups=3, act=2,
             last=False, p=0.25, unit="element", dtype="bf16"),
        # dropout into the residual stream of the widest layer configuration
        dict(name="drop 32x64x256^2 f16", op="drop", batch=32, channels=64, pixels=65536, last=False, residual=True,
             p=0.1, unit="element", dtype="f16"),
        # the smallest layer configuration, whole channels dropped: latency
        dict(name="drop 2x4x16^2 channel f32", op="drop", batch=2, channels=4, pixels=256, last=False, residual=True,
             p=0.5, unit="channel", dtype="f32"),
        # a conditioning or embedding stream; without a residual, as in a backward pass
        dict(name="drop 8192x1024 bf16", op="drop", batch=8192, channels=1024, pixels=1, last=False, residual=False,
             p=0.1, unit="element", dtype="bf16"),
        # a field of the network configuration in 4 bits
        dict(name="mx4_keep 20x64x256^2 f16", op="mx4_keep", batch=20, channels=64, pixels=65536, dtype="f16"),
        # wide mix of a token stream, both operands at hand: the largest product
        dict(name="mx4_mix 8192x4096x4096 bf16", op="mx4_mix", batch=8192, c_in=4096, c_out=4096, pixels=1, act=1,
             add=False, dtype="bf16"),
        # one token of a wide mix: bound by the weights' bytes
        dict(name="mx4_serve 1x8192x8192 bf16", op="mx4_serve", batch=1, c_in=8192, c_out=8192, pixels=1, act=0,
             add=False, dtype="bf16"),
        # ragged field: block's channel mix with the spectral branch added
        dict(name="mx4_serve 5x200x72x1001 f32", op="mx4_serve", batch=5, c_in=200, c_out=72, pixels=1001, act=1,
             add=True, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_step", "gn_step", "drop", "drop", "mx4_keep", "mx4_mix", "mx4_serve"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = (1 << 24) if dtype == "f32" else (1 << 25)  # elements of one field
    tokens = rng.random() < 0.35
    pixels = 1 if tokens else _log_int(rng, 2, 65536)
    if not tokens and rng.random() < 0.4:
        pixels = max(64, pixels // 64 * 64)  # power-of-two-like grids are the ordinary ones
    p = rng.choice([0.0, 0.1, 0.25, 0.5, 0.9])
    unit = rng.choice(["element", "element", "channel", "sample"])
    if op.startswith("gn"):
        groups = rng.choice([1, 2, 3, 4, 8, 16, 32])
        wide = _log_int(rng, 1, max(1, min(4096 if tokens else 512, most // pixels) // groups))
        if rng.random() < 0.5:
            wide = (wide + 7) // 8 * 8
        channels = groups * wide
        batch = _log_int(rng, 1, max(1, min(8192 if tokens else 32, most // (channels * pixels))))
        return dict(op=op, batch=batch, channels=channels, pixels=pixels, groups=groups, act=rng.choice([0, 1, 2]),
                    last=rng.random() < 0.5, p=p, unit=unit, dtype=dtype)
    channels = _log_int(rng, 1, 8192 if tokens else 512)
    batch = _log_int(rng, 1, max(1, min(8192 if tokens else 32, most // (channels * pixels))))
    if op == "drop":
        return dict(op=op, batch=batch, channels=channels, pixels=pixels, last=rng.random() < 0.5,
                    residual=rng.random() < 0.5, p=max(p, 0.1), unit=unit, dtype=dtype)
    if op == "mx4_keep":
        return dict(op=op, batch=batch, channels=channels, pixels=pixels, dtype=dtype)
    c_out = _log_int(rng, 1, 8192 if tokens else 512)
    if op == "mx4_serve" and rng.random() < 0.5:
        batch, pixels = rng.choice([1, 2, 3, 8]), 1
    batch = max(1, min(batch, most // (2 * pixels * max(channels, c_out)), (1 << 36) // (pixels * channels * c_out)))
    return dict(op=op, batch=batch, c_in=channels, c_out=c_out, pixels=pixels, act=rng.choice([0, 1]),
                add=rng.random() < 0.4, dtype=dtype)


def _packed_bytes(rows, n):
    return rows * -(-n // _BLOCK) * (_BLOCK // 2 + 1)


def work(case):
    s, op = _SIZE[case["dtype"]], case["op"]
    if op in ("mx4_mix", "mx4_serve"):
        ci, co, n = case["c_in"], case["c_out"], case["batch"] * case["pixels"]
        x = _packed_bytes(n, ci) if op == "mx4_mix" else s * n * ci
        return {"bytes": x + _packed_bytes(co, ci) + s * co + s * n * co * (2 if case["add"] else 1),
                "flops": 2 * n * ci * co}
    rows, n = case["batch"] * case["pixels"], case["batch"] * case["channels"] * case["pixels"]
    if op == "drop":
        return {"bytes": s * n * (3 if case["residual"] else 2), "flops": 2 * n}
    if op == "mx4_keep":
        return {"bytes": 2 * s * n + 2 * _packed_bytes(rows, case["channels"]), "flops": 2 * n}
    params = 2 * s * case["channels"]
    if op == "gn_fwd":
        return {"bytes": 2 * s * n + params, "flops": 10 * n}
    return {"bytes": 5 * s * n + 3 * params, "flops": 30 * n}


# ------------------------------------------------------------------ inputs

def _field(gen, shape, dtype, last=False, scale=1.0, mean=0.0):
    """A field [B][C][P] ([B][P][C] where last) whose channels differ in strength and level."""
    t = torch.randn(shape, generator=gen, device="cuda")
    per = (shape[0], 1, shape[2]) if last else (shape[0], shape[1], 1)
    r = torch.randn(per, generator=gen, device="cuda")
    t.mul_(scale * torch.exp(0.5 * r))
    if mean:
        t.add_(mean * torch.randn(per, generator=gen, device="cuda"))
    return t.to(_DT[dtype])


def _tokens(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(_DT[dtype])


def _pack(x):
    """(codes uint8 [rows][nb][32], exponents [rows][nb]) of x [rows][n] fp32: values
    of sign, two exponent bits and one mantissa bit, times 2^exponent a block."""
    rows, n = x.shape
    b = torch.nn.functional.pad(x, (0, -n % _BLOCK)).view(rows, -1, _BLOCK)
    m = b.abs().amax(-1)
    e = torch.where(m > 0, torch.frexp(m)[1] - 3, -127).clamp_(min=-127)
    v = torch.ldexp(b, -e.unsqueeze(-1)).abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = (v / step).round_().mul_(step).clamp_(max=6.0)  # 0 .5 1 1.5 2 3 4 6, ties to the even code
    code = torch.where(v < 2, 2 * v, torch.where(v < 4, v + 2, v / 2 + 4)).to(torch.uint8)
    return code + 8 * torch.signbit(b).to(torch.uint8), e


def _unpack(code, e, n):
    """The fp32 values that codes and exponents stand for, [rows][n]."""
    k = (code & 7).float()
    v = torch.where(k < 4, k / 2, torch.where(k < 6, k - 2, 2 * k - 8))
    v = torch.ldexp(torch.where(code >= 8, -v, v), e.unsqueeze(-1))
    return v.view(v.shape[0], -1)[:, :n]


def _write_packed(code, e):
    """The library's layout: two codes a byte (the even one low) [rows][16 nb], then
    from a multiple of 256 the exponents + 127 [rows][nb], to a multiple of 256."""
    q = (code[..., 0::2] | (code[..., 1::2] << 4)).reshape(-1)
    s = (e + 127).to(torch.uint8).reshape(-1)
    up = lambda n: (n + 255) // 256 * 256  # noqa: E731
    buf = torch.zeros(up(q.numel()) + up(s.numel()), dtype=torch.uint8, device=q.device)
    buf[:q.numel()] = q
    buf[up(q.numel()):up(q.numel()) + s.numel()] = s
    return buf


def _read_packed(buf, rows, n):
    nb = -(-n // _BLOCK)
    q = buf[:rows * nb * 16].view(rows, nb, 16)
    at = (rows * nb * 16 + 255) // 256 * 256
    code = torch.stack((q & 15, q >> 4), -1).view(rows, nb, _BLOCK)
    return code, buf[at:at + rows * nb].view(rows, nb).int() - 127


def _room(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    d, dt, op = case["dtype"], _DT[case["dtype"]], case["op"]
    B, P = case["batch"], case["pixels"]
    empty = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    st = {"case": case}
    if op in ("mx4_mix", "mx4_serve"):
        ci, co = case["c_in"], case["c_out"]
        A = _tokens(gen, (co, ci), "f32", 1 / math.sqrt(ci))
        st["A"] = _write_packed(*_pack(A))
        x = _field(gen, (B, ci, P), d)
        if P == 1:
            x = x.view(B, ci)
        if op == "mx4_mix":
            st["x"] = _write_packed(*_pack(x.float().view(B, ci, P).transpose(1, 2).reshape(B * P, ci)))
        else:
            st["x"], st["packed"] = x, _room(_packed_bytes(B * P, ci) + 512)
        shape = (B, co) if P == 1 else (B, co, P)
        st.update(bias=_tokens(gen, (co,), d, 0.1), add=_tokens(gen, shape, d) if case["add"] else None,
                  y=empty(*shape))
        return st
    C = case["channels"]
    last = case.get("last", False)
    shape = (B, P, C) if last else (B, C, P)
    flat = (B, C) if P == 1 else shape  # tokens
    if op == "mx4_keep":
        st.update(x=_field(gen, shape, d).view(flat), y=empty(*flat), packed=_room(_packed_bytes(B * P, C) + 512))
        return st
    st.update(p=case["p"], seed=int(torch.randint(1 << 62, (1,), generator=gen, device="cuda")),
              offset=int(torch.randint(1 << 40, (1,), generator=gen, device="cuda")))
    if op == "drop":
        st.update(v=_field(gen, shape, d, last).view(flat), y=empty(*flat),
                  x=_field(gen, shape, d, last).view(flat) if case["residual"] else None)
        return st
    G = case["groups"]
    near = lambda c, s, n: (c + s * torch.randn(n, generator=gen, device="cuda")).to(dt)  # noqa: E731
    st.update(x=_field(gen, shape, d, last, mean=0.5).view(flat), y=empty(*flat), weight=near(1.0, 0.2, (C,)),
              bias=near(0.0, 0.2, (C,)), stats=torch.empty((B, G, 2), dtype=torch.float32, device="cuda"),
              # sums per sample, channel and piece of its pixels
              workspace=_room(32 * B * C + (1 << 26)))
    if op == "gn_step":
        st.update(gy=_field(gen, shape, d, last, 0.02).view(flat), gx=empty(*flat), gw=empty(C), gb=empty(C))
    return st


# --------------------------------------------------------------- plain form

def _philox(block, seed, offset):
    """The four 32-bit words of the Philox 4x32-10 generator (Salmon, Moraes, Dror, Shaw:
    Parallel random numbers: as easy as 1, 2, 3, SC 2011) at 64-bit counters `block`
    (low half) and `offset` (high half), key `seed`; int64 tensors of values below 2^32."""
    c = [block & _LOW32, block >> 32, torch.full_like(block, offset & _LOW32), torch.full_like(block, offset >> 32)]
    k0, k1 = seed & _LOW32, seed >> 32
    for _ in range(10):
        # products below 2^64 in 64 signed bits: wrapped, their halves are right after masking
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & _LOW32) ^ c[1] ^ k0, b & _LOW32, ((a >> 32) & _LOW32) ^ c[3] ^ k1, a & _LOW32]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW32, (k1 + 0xBB67AE85) & _LOW32
    return c


def _threshold(p):
    return int(round(p * 65536))


def _keep_units(n, st):
    """Which of n units are kept: 16 bits each, eight units a block."""
    blocks = torch.arange(-(-n // 8), dtype=torch.int64, device="cuda")
    keep = torch.empty((blocks.numel(), 8), dtype=torch.bool, device="cuda")
    t = _threshold(st["p"])
    for i, w in enumerate(_philox(blocks, st["seed"], st["offset"])):
        keep[:, 2 * i] = (w & 0xFFFF) >= t
        keep[:, 2 * i + 1] = (w >> 16) >= t
    return keep.view(-1)[:n]


def _per_unit(keep, c):
    """A mask over units against [B][C][P] or [B][P][C]."""
    B, C, P = c["batch"], c["channels"], c["pixels"]
    if c["unit"] == "element":
        return keep.view((B, P, C) if c["last"] else (B, C, P))
    if c["unit"] == "channel":
        return keep.view((B, 1, C) if c["last"] else (B, C, 1))
    return keep.view(B, 1, 1)


def _units(c):
    return {"element": c["batch"] * c["channels"] * c["pixels"], "channel": c["batch"] * c["channels"],
            "sample": c["batch"]}[c["unit"]]


def _plain_drop(v, st, keep=None):
    """D(v) of a [B][C][P] / [B][P][C] fp32 tensor."""
    t = _threshold(st["p"])
    if t == 0:
        return v
    if keep is None:
        keep = _per_unit(_keep_units(_units(st["case"]), st), st["case"])
    return torch.where(keep, v * (65536.0 / (65536 - t) if t < 65536 else 0.0), 0.0)


def _act(z, act):
    if act == 1:
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-z)) if act == 2 else z


def _act_slope(z, act):
    if act == 1:
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == 2:
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def _grouped(t, c):
    """[B][G][C/G][P] or [B][P][G][C/G] view, and the axes of a group."""
    B, C, P, G = c["batch"], c["channels"], c["pixels"], c["groups"]
    return (t.view(B, P, G, C // G), (1, 3)) if c["last"] else (t.view(B, G, C // G, P), (2, 3))


def _per_channel(p, c):
    return p.float().view(1, 1, -1) if c["last"] else p.float().view(1, -1, 1)


def _run_plain_gn(st):
    c, dt = st["case"], st["x"].dtype
    B, C, P = c["batch"], c["channels"], c["pixels"]
    shape = (B, P, C) if c["last"] else (B, C, P)
    n = C // c["groups"] * P
    x, axes = _grouped(st["x"].float(), c)
    mean = (x.sum(axes, keepdim=True, dtype=torch.float64) / n).float()
    d = x - mean
    r = torch.rsqrt((d * d).sum(axes, keepdim=True, dtype=torch.float64) / n + _EPS).float()
    xh = (d * r).view(shape)
    z = xh * _per_channel(st["weight"], c) + _per_channel(st["bias"], c)
    keep = None
    if _threshold(c["p"]):
        keep = _per_unit(_keep_units(_units(c), st), c)
    out = {"y": _plain_drop(_act(z, c["act"]), st, keep).to(dt).view(st["x"].shape)}
    if c["op"] == "gn_fwd":
        return out
    gz = _plain_drop(st["gy"].float().view(shape), st, keep) * _act_slope(z, c["act"])
    over = (0, 1) if c["last"] else (0, 2)
    out["gw"] = (gz * xh).sum(over, dtype=torch.float64).to(dt)
    out["gb"] = gz.sum(over, dtype=torch.float64).to(dt)
    g, _ = _grouped(gz * _per_channel(st["weight"], c), c)
    h, _ = _grouped(xh, c)
    m1 = (g.sum(axes, keepdim=True, dtype=torch.float64) / n).float()
    m2 = ((g * h).sum(axes, keepdim=True, dtype=torch.float64) / n).float()
    out["gx"] = (r * (g - m1 - h * m2)).to(dt).view(st["x"].shape)
    return out


def _run_plain(st):
    c = st["case"]
    op = c["op"]
    if op.startswith("gn"):
        return _run_plain_gn(st)
    B, P = c["batch"], c["pixels"]
    if op == "drop":
        shape = (B, P, c["channels"]) if c["last"] else (B, c["channels"], P)
        y = _plain_drop(st["v"].float().view(shape), st).view(st["v"].shape)
        return {"y": (y if st["x"] is None else st["x"].float() + y).to(st["v"].dtype)}
    rows_of = lambda x, C: x.float().view(B, C, P).transpose(1, 2).reshape(B * P, C)  # noqa: E731
    if op == "mx4_keep":
        C, x = c["channels"], st["x"]
        v = _unpack(*_pack(rows_of(x, C)), C)
        return {"x": v.view(B, P, C).transpose(1, 2).to(x.dtype).reshape(x.shape)}
    ci, co = c["c_in"], c["c_out"]
    A = _unpack(*_read_packed(st["A"], co, ci), ci)
    x = _unpack(*(_read_packed(st["x"], B * P, ci) if op == "mx4_mix" else _pack(rows_of(st["x"], ci))), ci)
    z = torch.matmul(x, A.t()) + st["bias"].float()
    z = z.view(B, P, co).transpose(1, 2).reshape(st["y"].shape)
    if st["add"] is not None:
        z = z + st["add"].float()
    return {"y": _act(z, c["act"]).to(st["y"].dtype)}


# ---------------------------------------------------------------- own form

def _run_own(st):
    import spectral_convolution_amd as fno
    c = st["case"]
    op = c["op"]
    if op == "mx4_keep":
        fno.fno_mx4_pack(st["x"], st["packed"])
        fno.fno_mx4_unpack(st["packed"], st["y"])
        return {"x": st["y"]}
    if op in ("mx4_mix", "mx4_serve"):
        x = st["x"]
        if op == "mx4_serve":
            fno.fno_mx4_pack(x, st["packed"])
            x = st["packed"]
        fno.fno_channel_mix_mx4(x, st["A"], st["bias"], st["add"], st["y"], c["c_in"], act=c["act"])
        return {"y": st["y"]}
    drop = fno.Dropout(st["p"], st["seed"], st["offset"], unit=c["unit"]) if st["p"] > 0 else None
    if op == "drop":
        fno.fno_dropout_residual(drop, st["x"], st["v"], st["y"], channels_last=c["last"])
        return {"y": st["y"]}
    prm = fno.GroupNormParams(c["groups"], _EPS, st["weight"], st["bias"], act=c["act"], channels_last=c["last"])
    fno.fno_group_norm(prm, st["x"], st["y"], st["stats"], st["workspace"], dropout=drop)
    out = {"y": st["y"]}
    if op == "gn_step":
        fno.fno_group_norm_backward(prm, st["x"], st["stats"], st["gy"], st["gx"], st["gw"], st["gb"],
                                    st["workspace"], dropout=drop)
        out.update(gx=st["gx"], gw=st["gw"], gb=st["gb"])
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- exact

def _exact_bits(n, seed, offset):
    """16 random bits for each of n units: unit u has the halves of word (u % 8) / 2 of
    block u / 8. 32-bit words as pairs of 16-bit halves, so that no product passes 2^33."""
    def mul(w, m):  # (high word, low word) of w m, each a pair (low half, high half)
        ml, mh = m & 0xFFFF, m >> 16
        ll, lh, hl, hh = w[0] * ml, w[0] * mh, w[1] * ml, w[1] * mh
        mid = (ll >> 16) + (lh & 0xFFFF) + (hl & 0xFFFF)
        top = (mid >> 16) + (lh >> 16) + (hl >> 16) + (hh & 0xFFFF)
        return (top & 0xFFFF, (top >> 16) + (hh >> 16)), (ll & 0xFFFF, mid & 0xFFFF)

    def xor(a, b, k):
        return (a[0] ^ b[0] ^ (k & 0xFFFF), a[1] ^ b[1] ^ (k >> 16))

    i = torch.arange((n + 7) // 8, device="cuda")
    word = lambda v: tuple(torch.zeros_like(i) + ((v >> s) & 0xFFFF) for s in (0, 16))  # noqa: E731
    x0, x1, x2, x3 = word(i), word(i >> 32), word(offset), word(offset >> 32)
    for rnd in range(10):
        hi0, lo0 = mul(x0, 0xD2511F53)
        hi2, lo2 = mul(x2, 0xCD9E8D57)
        x0 = xor(hi2, x1, ((seed % 2 ** 32) + rnd * 0x9E3779B9) % 2 ** 32)
        x2 = xor(hi0, x3, ((seed // 2 ** 32) + rnd * 0xBB67AE85) % 2 ** 32)
        x1, x3 = lo2, lo0
    return torch.stack([h for w in (x0, x1, x2, x3) for h in w], 1).reshape(-1)[:n]


def _exact_drop_factor(c, st):
    """The factor of D(v), against [B][C][P] / [B][P][C], or None where nothing is dropped."""
    t = round(c["p"] * 65536)
    if t == 0:
        return None
    B, C, P = c["batch"], c["channels"], c["pixels"]
    shape = {"element": (B, P, C) if c["last"] else (B, C, P),
             "channel": (B, 1, C) if c["last"] else (B, C, 1), "sample": (B, 1, 1)}[c["unit"]]
    bits = _exact_bits(math.prod(shape), st["seed"], st["offset"]).view(shape)
    return torch.where(bits < t, 0.0, 65536.0 / max(65536 - t, 1)).double()


def _exact_trip(rows):
    """The 4-bit values of rows [n][C] in fp64: the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 times the block's
    power of two, the one with the even code where two are as near."""
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=rows.device)
    borders = (grid[1:] + grid[:-1]) / 2
    n, C = rows.shape
    b = torch.nn.functional.pad(rows.double(), (0, -C % 32)).unflatten(-1, (-1, 32))
    top = b.abs().max(-1, keepdim=True).values
    power = (torch.frexp(top).exponent.double() - 3).masked_fill(top == 0, 0).clamp(min=-127)
    v = b.abs() / torch.exp2(power)
    low = torch.bucketize(v, borders)                 # a tie stays with the lower one here
    high = torch.bucketize(v, borders, right=True)    # and goes to the upper one here
    code = torch.where(low % 2 == 0, low, high)
    return (torch.sign(b) * grid[code] * torch.exp2(power)).flatten(-2)[:, :C]


def exact(case, seed):
    st = prepare(case, seed)
    op, B, P = case["op"], case["batch"], case["pixels"]
    if op == "mx4_keep":
        C = case["channels"]
        rows = st["x"].reshape(B, C, P).permute(0, 2, 1).reshape(-1, C)
        return {"x": _exact_trip(rows).view(B, P, C).permute(0, 2, 1).reshape(st["x"].shape)}
    if op.startswith("mx4"):
        ci, co = case["c_in"], case["c_out"]
        gen = torch.Generator(device="cuda").manual_seed(int(seed))  # the values behind the packed operands
        A = _exact_trip(_tokens(gen, (co, ci), "f32", 1 / math.sqrt(ci)))
        x = _exact_trip(_field(gen, (B, ci, P), case["dtype"]).permute(0, 2, 1).reshape(-1, ci))
        z = (x @ A.t() + st["bias"].double()).view(B, P, co).permute(0, 2, 1).reshape(st["y"].shape)
        if st["add"] is not None:
            z = z + st["add"].double()
        return {"y": z * torch.special.ndtr(z) if case["act"] else z}
    C = case["channels"]
    shape = (B, P, C) if case["last"] else (B, C, P)
    factor = _exact_drop_factor(case, st)
    if op == "drop":
        y = st["v"].double().reshape(shape)
        y = (y if factor is None else y * factor).reshape(st["v"].shape)
        return {"y": y if st["x"] is None else y + st["x"].double()}
    G = case["groups"]
    leaves = [st[k].double().requires_grad_(op == "gn_step") for k in ("x", "weight", "bias")]
    x, w, b = leaves
    at = (lambda p: p.view(1, 1, C)) if case["last"] else (lambda p: p.view(1, C, 1))
    h = x.reshape(B, P, G, C // G) if case["last"] else x.reshape(B, G, C // G, P)
    over = (1, 3) if case["last"] else (2, 3)
    size = C // G * P
    h = h - h.sum(over, keepdim=True) / size
    h = h / torch.sqrt(h.square().sum(over, keepdim=True) / size + _EPS)
    z = h.reshape(shape) * at(w) + at(b)
    y = [z, z * torch.special.ndtr(z), z * torch.sigmoid(z)][case["act"]]
    y = (y if factor is None else y * factor).reshape(st["x"].shape)
    out = {"y": y.detach()}
    if op == "gn_step":
        out.update(zip(("gx", "gw", "gb"), torch.autograd.grad(y, leaves, st["gy"].double())))
    return out
