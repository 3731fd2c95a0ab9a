"""Cases of the training operators around an FNO block: the 8-bit activation
checkpoints, the channel mix that keeps them and its backward pass, and the
norms before and after a block with its gate and residual scale.

Fields are [batch][channels][pixels]. With `own` true run() calls the
library; otherwise it computes the same outputs with elementary torch
operations in fp32 (fp64 for sums over pixels), rounded once at the end.
exact() computes them in fp64 from the definitions, gradients by automatic
differentiation.

Operators ("op" of a case):
  checkpoint  pack a field into 8 bits and unpack it again
  mix_step    channel mix that keeps its checkpoints, then the backward from them
  mix_bwd     that backward alone, the checkpoints at hand
  norm_fwd    y = x + scale gate N(v), u = N'(y)
  norm_bwd    its backward from the stored fields
  norm_step   the forward that keeps checkpoints, then the backward from them
"""

import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5
_BLOCK = 32  # values that share one exponent


# ------------------------------------------------------------------- cases

def listed():
    return [
        # residual glue of the widest layer configuration: 64 channels of 256 x 256, batch 32
        dict(name="norm_fwd 32x64x256^2 f16", op="norm_fwd", batch=32, channels=64, pixels=65536, dtype="f16",
             kind="rms"),
        # the smallest layer configuration (16 x 16, 4 channels): a call's latency
        dict(name="norm_fwd 2x4x16^2 f32", op="norm_fwd", batch=2, channels=4, pixels=256, dtype="f32", kind="rms"),
        # token layout (one pixel): a conditioning or embedding stream
        dict(name="norm_fwd 8192x1024 bf16", op="norm_fwd", batch=8192, channels=1024, pixels=1, dtype="bf16",
             kind="layer"),
        # training of the 64^3 configuration, fp32, fields kept whole
        dict(name="norm_bwd 4x32x64^3 f32", op="norm_bwd", batch=4, channels=32, pixels=262144, dtype="f32",
             kind="layer"),
        # training step of the network configuration, fields kept in 8 bits
        dict(name="norm_step 20x64x256^2 f16", op="norm_step", batch=20, channels=64, pixels=65536, dtype="f16",
             kind="rms"),
        # ragged: 61 x 61 grid, 48 channels
        dict(name="norm_step 3x48x61^2 bf16", op="norm_step", batch=3, channels=48, pixels=3721, dtype="bf16",
             kind="layer"),
        # training step of the widest layer configuration's bypass: the largest case
        dict(name="mix_step 32x64x64x256^2 f16", op="mix_step", batch=32, c_in=64, c_out=64, pixels=65536,
             dtype="f16", act=1, add=True),
        # the 128 x 128 configuration in fp32
        dict(name="mix_step 16x32x32x128^2 f32", op="mix_step", batch=16, c_in=32, c_out=32, pixels=16384,
             dtype="f32", act=1, add=True),
        # ragged: odd channel counts and a pixel count that is no multiple of anything
        dict(name="mix_step 5x40x72x1001 bf16", op="mix_step", batch=5, c_in=40, c_out=72, pixels=1001, dtype="bf16",
             act=1, add=False),
        # the smallest configuration's backward: latency
        dict(name="mix_bwd 2x4x4x16^2 f32", op="mix_bwd", batch=2, c_in=4, c_out=4, pixels=256, dtype="f32", act=1,
             add=True),
        # a field of the network configuration kept in 8 bits
        dict(name="checkpoint 1280x256^2 bf16", op="checkpoint", rows=1280, pixels=65536, dtype="bf16"),
        # ragged rows in fp32
        dict(name="checkpoint 96x3721 f32", op="checkpoint", rows=96, pixels=3721, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_step", "mix_step", "mix_bwd", "checkpoint"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    most = (1 << 25) if dtype == "f32" else (1 << 26)  # elements of one field
    pixels = _log_int(rng, 33, 65536)
    if rng.random() < 0.4:
        pixels = max(64, pixels // 64 * 64)  # power-of-two-like grids are the ordinary ones
    if op == "checkpoint":
        return dict(op=op, rows=_log_int(rng, 1, min(4096, max(1, most // pixels))), pixels=pixels, dtype=dtype)
    if op.startswith("mix"):
        c_in, c_out = _log_int(rng, 1, 128), _log_int(rng, 1, 128)
        batch = _log_int(rng, 1, max(1, min(32, (most // 2) // (max(c_in, c_out) * pixels))))
        return dict(op=op, batch=batch, c_in=c_in, c_out=c_out, pixels=pixels, dtype=dtype, act=rng.choice([0, 1, 1]),
                    add=rng.random() < 0.6)
    kind = rng.choice(["rms", "layer"])
    if op != "norm_step" and rng.random() < 0.35:  # token layout
        channels = _log_int(rng, 16, 8192)
        return dict(op=op, batch=_log_int(rng, 1, min(16384, (most // 2) // channels)), channels=channels, pixels=1,
                    dtype=dtype, kind=kind)
    channels = _log_int(rng, 8, 256)
    return dict(op=op, batch=_log_int(rng, 1, max(1, min(32, most // (channels * pixels)))), channels=channels,
                pixels=pixels, dtype=dtype, kind=kind)


def work(case):
    s = _SIZE[case["dtype"]]
    q = 1 + 1 / _BLOCK  # bytes of one checkpointed value
    if case["op"] == "checkpoint":
        n = case["rows"] * case["pixels"]
        return {"bytes": n * (2 * s + 2 * q), "flops": 2 * n}
    if case["op"].startswith("mix"):
        ci, co, n = case["c_in"], case["c_out"], case["batch"] * case["pixels"]
        kept = ci + (co if case["act"] and case["add"] else 0)
        bwd = n * (s * (ci + co + (co if case["add"] else 0)) + q * kept) + 2 * s * ci * co
        products = 3 if case["act"] else 2
        if case["op"] == "mix_bwd":
            return {"bytes": bwd, "flops": 2 * products * n * ci * co}
        fwd = n * (s * (ci + co + (co if case["add"] else 0)) + q * kept) + s * ci * co
        return {"bytes": fwd + bwd, "flops": 2 * (products + 1) * n * ci * co}
    n = case["batch"] * case["channels"] * case["pixels"]
    gate = 2 * s * case["batch"] * case["channels"]
    if case["op"] == "norm_fwd":
        return {"bytes": 4 * s * n + gate / 2, "flops": 12 * n}
    if case["op"] == "norm_bwd":
        return {"bytes": 6 * s * n + gate, "flops": 30 * n}
    return {"bytes": 4 * s * n + 2 * q * n + 4 * s * n + 2 * q * n + 1.5 * gate, "flops": 42 * n}


# ------------------------------------------------------------------ inputs

def _field(gen, shape, dtype, scale=1.0):
    """A field whose rows (last axis) differ in strength, as channels do."""
    t = torch.randn(shape, generator=gen, device="cuda")
    r = torch.randn(shape[:-1] + (1,), generator=gen, device="cuda")
    return t.mul_(scale * torch.exp(0.5 * r)).to(_DT[dtype])


def _tokens(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(_DT[dtype])


def _checkpoint_of(x):
    """(codes int8 [rows][padded length], exponents int8 [rows][blocks]) of x
    [rows][length], as the library's checkpoint format defines them."""
    rows, n = x.shape
    pad = -n % _BLOCK
    b = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, _BLOCK)
    m = b.abs().amax(-1)
    low = -24 if x.dtype == torch.float16 else -126
    e = torch.where(m > 0, torch.frexp(m)[1] - 7, low).clamp_(min=low)
    # two factors: 2^126 alone is the largest power whose inverse is normal
    q = torch.ldexp(torch.ldexp(b, -(e // 2).unsqueeze(-1)), -(e - e // 2).unsqueeze(-1))
    q = q.round_().clamp_(-127, 127)
    bad = ~torch.isfinite(m)
    e = torch.where(bad, 127, e)
    q = torch.where(bad.unsqueeze(-1), 0.0, q)
    return q.to(torch.int8).view(rows, -1), e.to(torch.int8)


def _values_of(codes, exps, n):
    """The fp32 values that codes and exponents stand for, [rows][n]."""
    rows = codes.shape[0]
    v = torch.ldexp(codes.float().view(rows, -1, _BLOCK), exps.int().unsqueeze(-1))
    v = torch.where((exps == 127).unsqueeze(-1), float("nan"), v)
    return v.view(rows, -1)[:, :n]


def _round_trip(x):
    """x^ of a field [..., pixels] in fp32."""
    flat = x.reshape(-1, x.shape[-1])
    return _values_of(*_checkpoint_of(flat), flat.shape[1]).view(x.shape)


def _write_checkpoint(buf, at, x):
    """Lay the checkpoint of x [rows][length] out in `buf` from byte `at`;
    returns the byte after it (each part starts on a multiple of 256)."""
    for part in _checkpoint_of(x):
        n = part.numel()
        buf[at:at + n] = part.reshape(-1).view(torch.uint8)
        at += (n + 255) // 256 * 256
    return at


def _checkpoint_bytes(rows, n):
    nb = (n + _BLOCK - 1) // _BLOCK
    return (rows * nb * _BLOCK + 255) // 256 * 256 + (rows * nb + 255) // 256 * 256


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DT[case["dtype"]]
    d = case["dtype"]
    empty = lambda *shape: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
    room = lambda n: torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")  # noqa: E731
    st = {"case": case}
    if case["op"] == "checkpoint":
        rows, n = case["rows"], case["pixels"]
        st.update(x=_field(gen, (rows, n), d), out=empty(rows, n), saved=room(_checkpoint_bytes(rows, n)))
        return st
    B, P = case["batch"], case["pixels"]
    if case["op"].startswith("mix"):
        ci, co = case["c_in"], case["c_out"]
        x = _field(gen, (B, ci, P), d)
        add = _field(gen, (B, co, P), d) if case["add"] else None
        keep_add = case["add"] and case["act"]
        st.update(A=_tokens(gen, (co, ci), d, 1 / math.sqrt(ci)), bias=_tokens(gen, (co,), d, 0.1),
                  gy=_field(gen, (B, co, P), d, 0.02), gx=empty(B, ci, P), gA=empty(co, ci), gbias=empty(co),
                  gadd=empty(B, co, P) if case["add"] else None,
                  saved=room(_checkpoint_bytes(B * ci, P) + (_checkpoint_bytes(B * co, P) if keep_add else 0)),
                  # partial sums of the weight gradient: one [co][ci] matrix and one bias row per workgroup
                  workspace=room(1024 * 4 * (co * ci + co)))
        if case["op"] == "mix_bwd":
            at = _write_checkpoint(st["saved"], 0, x.view(B * ci, P))
            if keep_add:
                _write_checkpoint(st["saved"], at, add.view(B * co, P))
        else:
            st.update(x=x, add=add, y=empty(B, co, P))
        return st
    C = case["channels"]
    make = _field if P > 1 else _tokens
    shape = (B, C, P) if P > 1 else (B, C)
    near = lambda c, s, n: (c + s * torch.randn(n, generator=gen, device="cuda")).to(dt)  # noqa: E731
    layer = case["kind"] == "layer"
    st.update(x=make(gen, shape, d), v=make(gen, shape, d, 3.0), y=empty(*shape), u=empty(*shape),
              w_post=near(1.0, 0.2, (C,)), b_post=near(0.0, 0.1, (C,)) if layer else None,
              gate=near(0.5, 0.3, (B, C)), scale=near(0.2, 0.05, (C,)),
              w_pre=near(1.0, 0.2, (C,)), b_pre=near(0.0, 0.1, (C,)) if layer else None)
    if case["op"] != "norm_fwd":
        st.update(gy=make(gen, shape, d, 0.02), gu=make(gen, shape, d, 0.02), gx=empty(*shape), gv=empty(*shape),
                  # partial sums per workgroup and channel
                  workspace=room(4 * 4 * C * (4096 + 2 * B)))
        st["grads"] = {k: torch.empty_like(st[k]) for k in _NORM_PARAMS if st[k] is not None}
    if case["op"] == "norm_step":
        st["saved"] = room(2 * _checkpoint_bytes(B * C, P))
    return st


_NORM_PARAMS = ("w_post", "b_post", "gate", "scale", "w_pre", "b_pre")


# --------------------------------------------------------------- plain form

def _gelu(z):
    return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))


def _gelu_slope(z):
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))


def _plain_mix(A, bias, x, add):
    z = torch.matmul(A, x) + bias[:, None]
    return z if add is None else z + add


def _plain_mix_backward(st, xh, addh):
    """Gradients of the channel mix at the checkpointed inputs."""
    c, dt = st["case"], st["gy"].dtype
    A, bias, gz = st["A"].float(), st["bias"].float(), st["gy"].float()
    if c["act"]:
        gz = gz * _gelu_slope(_plain_mix(A, bias, xh, addh))
    out = {"gx": torch.matmul(A.t().contiguous(), gz).to(dt),
           "gA": torch.matmul(gz, xh.transpose(1, 2).contiguous()).sum(0, dtype=torch.float64).to(dt),
           "gbias": gz.sum((0, 2), dtype=torch.float64).to(dt)}
    if c["add"]:
        out["gadd"] = gz.to(dt)
    return out


def _stats(v, kind):
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    return d, torch.rsqrt((d * d).mean(1, keepdim=True) + _EPS)


def _col(p, ndim):
    """A per-channel [C] or per-sample [B][C] parameter against [B][C](...)."""
    p = p.float() if p.dim() == 2 else p.float()[None]
    return p if ndim == 2 else p[..., None]


def _plain_norm(st, x, v):
    """y and u in fp32."""
    k, nd = st["case"]["kind"], x.dim()
    at = lambda name: 0.0 if st[name] is None else _col(st[name], nd)  # noqa: E731
    d, r = _stats(v, k)
    y = x + at("scale") * at("gate") * (d * r * at("w_post") + at("b_post"))
    e, ry = _stats(y, k)
    return y, e * ry * at("w_pre") + at("b_pre")


def _norm_slope(g, vh, r, kind):
    """Gradient through vh = (v - mean) r at g = dL/dvh."""
    t = g - vh * (g * vh).mean(1, keepdim=True)
    return r * (t - g.mean(1, keepdim=True) if kind == "layer" else t)


def _plain_norm_backward(st, x, v):
    k, nd, dt = st["case"]["kind"], x.dim(), st["gy"].dtype
    at = lambda name: 0.0 if st[name] is None else _col(st[name], nd)  # noqa: E731
    over_p = lambda t: t.sum(2, dtype=torch.float64) if nd == 3 else t.double()  # noqa: E731
    d, r = _stats(v, k)
    vh = d * r
    n = vh * at("w_post") + at("b_post")
    e, ry = _stats(x + at("scale") * at("gate") * n, k)
    yh = e * ry
    gu = st["gu"].float()
    gy = st["gy"].float() + _norm_slope(gu * at("w_pre"), yh, ry, k)
    gn = gy * at("scale") * at("gate")
    out = {"gx": gy.to(dt), "gv": _norm_slope(gn * at("w_post"), vh, r, k).to(dt),
           "g_gate": over_p(gy * at("scale") * n).to(dt),
           "g_scale": over_p(gy * at("gate") * n).sum(0).to(dt),
           "g_w_post": over_p(gn * vh).sum(0).to(dt), "g_w_pre": over_p(gu * yh).sum(0).to(dt)}
    if st["b_post"] is not None:
        out["g_b_post"] = over_p(gn).sum(0).to(dt)
        out["g_b_pre"] = over_p(gu).sum(0).to(dt)
    return out


def _run_plain(st):
    c = st["case"]
    op, n = c["op"], c["pixels"]
    if op == "checkpoint":
        return {"x": _values_of(*_checkpoint_of(st["x"]), n).to(st["x"].dtype)}
    if op == "mix_bwd":
        B, ci, co = c["batch"], c["c_in"], c["c_out"]
        nb = (n + _BLOCK - 1) // _BLOCK

        def read(at, rows):
            q = st["saved"][at:at + rows * nb * _BLOCK].view(torch.int8).view(rows, -1)
            at += (rows * nb * _BLOCK + 255) // 256 * 256
            e = st["saved"][at:at + rows * nb].view(torch.int8).view(rows, -1)
            return _values_of(q, e, n)

        xh = read(0, B * ci).view(B, ci, n)
        addh = read(_checkpoint_bytes(B * ci, n), B * co).view(B, co, n) if c["add"] and c["act"] else None
        return _plain_mix_backward(st, xh, addh)
    if op == "mix_step":
        add = None if st["add"] is None else st["add"].float()
        z = _plain_mix(st["A"].float(), st["bias"].float(), st["x"].float(), add)
        y = (_gelu(z) if c["act"] else z).to(st["x"].dtype)
        addh = _round_trip(st["add"]) if c["add"] and c["act"] else None
        return {"y": y, **_plain_mix_backward(st, _round_trip(st["x"]), addh)}
    dt = st["x"].dtype
    x, v = st["x"].float(), st["v"].float()
    if op == "norm_bwd":
        return _plain_norm_backward(st, x, v)
    y, u = _plain_norm(st, x, v)
    out = {"y": y.to(dt), "u": u.to(dt)}
    if op == "norm_step":
        out.update(_plain_norm_backward(st, _round_trip(st["x"]), _round_trip(st["v"])))
    return out


# ---------------------------------------------------------------- own form

def _own_mix_backward(fno, st):
    c = st["case"]
    fno.fno_channel_mix_backward_saved(st["saved"], st["A"], st["bias"], st["gy"], st["gx"], st["gA"], st["gbias"],
                                       st["gadd"], st["workspace"], act=c["act"], has_add=c["add"])
    out = {"gx": st["gx"], "gA": st["gA"], "gbias": st["gbias"]}
    if c["add"]:
        out["gadd"] = st["gadd"]
    return out


def _run_own(st):
    import spectral_convolution_amd as fno
    c = st["case"]
    op = c["op"]
    if op == "checkpoint":
        fno.fno_checkpoint_pack(st["x"], st["saved"])
        fno.fno_checkpoint_unpack(st["saved"], st["out"])
        return {"x": st["out"]}
    if op == "mix_bwd":
        return _own_mix_backward(fno, st)
    if op == "mix_step":
        fno.fno_channel_mix_save(st["x"], st["A"], st["bias"], st["add"], st["y"], st["saved"], act=c["act"])
        return {"y": st["y"], **_own_mix_backward(fno, st)}
    prm = fno.NormParams(c["kind"], _EPS, **{k: st[k] for k in _NORM_PARAMS})
    out = {}
    if op == "norm_fwd":
        fno.fno_norm_residual(prm, st["x"], st["v"], st["y"], st["u"])
        return {"y": st["y"], "u": st["u"]}
    grads = fno.NormGrads(**st["grads"])
    if op == "norm_bwd":
        fno.fno_norm_residual_backward(prm, st["x"], st["v"], st["gy"], st["gu"], st["gx"], st["gv"], grads,
                                       st["workspace"])
    else:
        fno.fno_norm_residual_save(prm, st["x"], st["v"], st["y"], st["u"], st["saved"])
        fno.fno_norm_residual_backward_saved(prm, st["saved"], st["gy"], st["gu"], st["gx"], st["gv"], grads,
                                             st["workspace"])
        out.update(y=st["y"], u=st["u"])
    out.update(gx=st["gx"], gv=st["gv"], **{"g_" + k: t for k, t in st["grads"].items()})
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- exact

def _exact_trip(x):
    """The checkpointed values of x [..., n] in fp64: per block of 32, the
    nearest multiples of 2^(floor(log2 max) - 6), at most 127 of them."""
    n = x.shape[-1]
    blocks = torch.nn.functional.pad(x.double(), (0, -n % 32)).unflatten(-1, (-1, 32))
    top = blocks.abs().max(-1, keepdim=True).values
    # frexp: top = f 2^k with f in [1/2, 1), so floor(log2 top) = k - 1
    power = torch.frexp(top).exponent.double() - 1 - 6
    power = power.masked_fill(top == 0, 0).clamp(min=-24 if x.dtype == torch.float16 else -126)
    step = torch.exp2(power)
    return (torch.round(blocks / step).clamp(-127, 127) * step).flatten(-2)[..., :n]


def _exact_norm(t, w, b, kind):
    if kind == "layer":
        t = t - t.sum(1, keepdim=True) / t.shape[1]
    t = t / torch.sqrt(t.square().sum(1, keepdim=True) / t.shape[1] + _EPS) * w
    return t if b is None else t + b


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        return {"x": _exact_trip(st["x"])}
    if op.startswith("mix"):
        if op == "mix_bwd":  # the fields behind the checkpoints, made again
            whole = prepare(dict(case, op="mix_step"), seed)
        else:
            whole = st

        def mix(x, A, bias, add):
            z = torch.einsum("oi,bip->bop", A, x) + bias.view(1, -1, 1)
            z = z if add is None else z + add
            return z * torch.special.ndtr(z) if case["act"] else z

        A, bias, x = st["A"].double(), st["bias"].double(), whole["x"]
        add = whole["add"]
        out = {}
        if op == "mix_step":
            out["y"] = mix(x.double(), A, bias, None if add is None else add.double())
        leaves = [_exact_trip(x).requires_grad_(), A.requires_grad_(), bias.requires_grad_()]
        if add is not None:
            leaves.append(_exact_trip(add).requires_grad_())
        got = torch.autograd.grad(mix(*leaves[:3], leaves[3] if add is not None else None), leaves, st["gy"].double())
        out.update(zip(("gx", "gA", "gbias", "gadd"), got))
        return out
    kind = case["kind"]
    spread = lambda p: None if p is None else p.double().reshape(  # noqa: E731
        (p.shape if p.dim() == 2 else (1,) + p.shape) + (1,) * (st["x"].dim() - 2))
    names = [k for k in _NORM_PARAMS if st[k] is not None]
    p = {k: spread(st[k]) for k in _NORM_PARAMS}

    def both(x, v):
        y = x + p["scale"] * p["gate"] * _exact_norm(v, p["w_post"], p["b_post"], kind)
        return y, _exact_norm(y, p["w_pre"], p["b_pre"], kind)

    out = {}
    if op != "norm_bwd":
        out["y"], out["u"] = both(st["x"].double(), st["v"].double())
    if op == "norm_fwd":
        return out
    at = _exact_trip if op == "norm_step" else torch.Tensor.double
    x, v = at(st["x"]).requires_grad_(), at(st["v"]).requires_grad_()
    for k in names:
        p[k].requires_grad_()
    got = torch.autograd.grad(both(x, v), [x, v] + [p[k] for k in names], (st["gy"].double(), st["gu"].double()))
    out.update(gx=got[0], gv=got[1], **{"g_" + k: g.reshape(st[k].shape) for k, g in zip(names, got[2:])})
    return out
