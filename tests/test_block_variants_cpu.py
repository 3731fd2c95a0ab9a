"""The shapes of the block operators' GPU tests launch every one of their kernels: the library's host
code runs on the CPU against the recording runtime, which names the kernels (csrc/check)."""

import os
import re
import shutil

import pytest

import test_gpu_dropout as drop
import test_gpu_group_norm as gnorm
import test_gpu_mx4 as mx4
from spectral_convolution_amd import bounds_check
from test_training_variants_cpu import _program

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="needs hipcc (host-only compile)")
OWN = re.compile(r"fno::(fno_(?:gnorm|drop|mx4)\w*<[^>]*>)")


def _kernels(args, calls=()):
    r = bounds_check.run(_program(), args=args, calls="\n".join(calls) + "\n")
    assert r.returncode == 0, r.stderr[-2000:]
    return {m.group(1) for m in map(OWN.search, r.stdout.splitlines()) if m}


def test_every_kernel_is_reached():
    calls = []
    for d in range(3):
        calls += [f"gnorm {d} {B} {C} {P} {G} {last}" for B, C, P, G in gnorm.SHAPES for last in (0, 1)]
        calls += [f"drop {d} {B} {C} {P}" for B, C, P in drop.SHAPES]
        calls += [f"mx4 {d} {B} {I} {O} {P}" for B, I, O, P in mx4.MIXES]
        calls += [f"mx4 {d} {B} {I} {O} 1" for B, O, I in mx4.LARGE]
    have, ran = _kernels(["kernels"]), _kernels(["trace"], calls)
    assert len(have) > 100 and have - ran == set()
