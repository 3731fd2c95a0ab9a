"""The shapes of tests/test_gpu_training_variants.py launch every kernel of the training
operators, with more than one tile or row a workgroup: the library's host code runs on the CPU
against the recording runtime, which names the kernels (csrc/check)."""

import os
import re
import shutil

import pytest

import training_ref64 as r64
from spectral_convolution_amd import bounds_check

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="needs hipcc (host-only compile)")
CODE = {"f32": 0, "f16": 1, "bf16": 2}
OWN = re.compile(r"fno::(fno_(?:norm|mix|checkpoint)\w*<[^>]*>)")


def _program():
    prog = os.path.join(bounds_check.OUT, "fno_bounds_check")
    src = [os.path.join(d, f) for d in (bounds_check.CSRC, os.path.join(bounds_check.CSRC, "check")) for f in os.listdir(d)]
    newest = max(os.path.getmtime(f) for f in src if os.path.isfile(f))
    return prog if os.path.exists(prog) and os.path.getmtime(prog) > newest else bounds_check.build()


def _launches(calls):
    r = bounds_check.run(_program(), args=["trace"], calls="\n".join(calls) + "\n")
    assert r.returncode == 0, r.stderr[-2000:]
    rows = [line.split(" | ") for line in r.stdout.splitlines()]
    return [(OWN.search(k).group(1), *map(int, g.split())) for k, g in rows if OWN.search(k)]


def _fields(shapes):
    return [f"norm {CODE[d]} {kind} {B} {C} {P}" for d in CODE for kind in (0, 1) for B, C, P in shapes(d)]


def _shapes():
    few = _fields(lambda d: [r64.few(C, d) for C in r64.FEW_CHANNELS])
    many = _fields(lambda d: [r64.many(C, d) for C in r64.SMALL_CHANNELS + r64.MANY_CHANNELS])
    tokens = _fields(lambda d: [(rows, C, 1) for C, rows in r64.TOKENS[d]])
    mix = [f"mix {CODE[d]} {r64.mix_many(O, d)[0]} {I} {O} {r64.mix_many(O, d)[1]} 1 1"
           for d in CODE for O in r64.MIX_CHANNELS for I in r64.MIX_CHANNELS]
    return few, many, tokens, mix


def test_every_kernel_is_reached():
    few, many, tokens, mix = _shapes()
    ran = {k for k, *_ in _launches(few + many + tokens + mix + [f"checkpoint {d} 5 40" for d in range(3)])}
    r = bounds_check.run(_program(), args=["kernels"])
    have = {m.group(1) for m in map(OWN.search, r.stdout.splitlines()) if m}
    assert len(have) > 300 and have - ran == set()


def test_workgroups_have_several_tiles():
    _, many, tokens, mix = _shapes()
    for calls in (many, tokens, mix):
        got = iter(_launches(calls))
        for call in calls:
            op, *a = call.split()
            dt, *a = map(int, a)
            for k, gx, gy, threads in (next(got), next(got), next(got)):
                if "_params" in k:
                    continue
                args = [int(v) if v.isdigit() else v for v in k[k.index("<") + 1:-1].split(", ")]
                if op == "mix":
                    B, P = a[0], a[3]
                    # the kernels' tiles: 64 pixels for each of the waves beside those of c_out
                    waves = threads // 64
                    O = args[-2]
                    tiles = B * -(-P // (64 * waves // O))
                    assert tiles >= 2 * gx, (call, k, gx)
                    continue
                kind, B, C, P = a
                if P == 1:
                    slots = gx * max(1, threads // args[1])  # args: type, threads of a row, pieces, kind
                    assert B > slots, (call, k, gx)
                else:
                    px = r64.field_tile("f32" if dt == 0 else "f16")
                    at_once = (threads // 64) // args[2]     # args: type, channels a lane, waves a tile, kind
                    per = -(-(-(-P // px)) // gx)
                    assert per > at_once and P % px, (call, k, gx)
        assert next(got, None) is None
