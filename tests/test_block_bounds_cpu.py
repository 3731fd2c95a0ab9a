"""The loads and stores of the block operators' kernels stay inside their buffers: the library's host code
runs on the CPU against the recording runtime, where every launcher states what its kernel reads and writes as
the kernel indexes it (csrc/check)."""

import os
import shutil

import pytest

from spectral_convolution_amd import bounds_check
from test_training_variants_cpu import _program

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="needs hipcc (host-only compile)")


def _trace(*calls):
    r = bounds_check.run(_program(), args=["trace"], calls="\n".join(calls) + "\n")
    assert "bounds:" not in r.stderr, r.stderr[-2000:]
    assert r.returncode == 0, r.stdout[-500:] + r.stderr[-2000:]
    return r.stdout


# (B, C, P, groups): rows that end inside 16 bytes, fewer chunks a group than its team has room for, in teams of 8, 16,
# 64, 256 and 1024 lanes, so that the field ends with a chunk that lanes without one load too
RAGGED = [(32, 64, 9, 16), (97, 61, 97, 1), (2, 48, 33, 3), (3, 33, 1, 3), (9, 257, 1, 1), (61, 2048, 1, 2048 // 32),
          (1, 4096, 61, 64), (97, 130, 57, 1), (100, 700, 41, 1)]


@pytest.mark.parametrize("shape", RAGGED, ids=str)
def test_small_groups_are_read_inside_the_field(shape):
    B, C, P, G = shape
    for d in range(3):
        for last in (0, 1):
            out = _trace(f"gnorm {d} {B} {C} {P} {G} {last}")
            assert "fno_gnorm_small" in out


# channels last and groups past a team's registers: rows that end inside 16 bytes, up to the field's end
COLUMNS = [(5, 61, 20000, 1), (5, 4, 56935, 2), (1, 3, 90001, 1), (1, 2057, 9001, 1), (2, 8191, 65537, 1)]


@pytest.mark.parametrize("shape", COLUMNS, ids=str)
def test_large_groups_are_read_inside_the_field(shape):
    B, C, P, G = shape
    for d in range(3):
        out = _trace(f"gnorm {d} {B} {C} {P} {G} 1", f"gnorm {d} {B} {C} {P} {G} 0")
        assert "fno_gnorm_cols" in out and "fno_gnorm_rows" in out


@pytest.mark.parametrize("shape", [(3, 7, 33), (15, 189, 2622), (2000, 3, 3), (1, 37, 5000), (7, 130, 9), (1, 1, 1)], ids=str)
def test_dropout_reads_inside_the_field(shape):
    _trace(*(f"drop {d} {' '.join(map(str, shape))}" for d in range(3)))


@pytest.mark.parametrize("shape", [(1, 8192, 8192, 1), (3, 1100, 70, 1), (1, 4001, 300, 1), (20, 1024, 31, 1), (2, 1056, 16, 33)], ids=str)
def test_few_rows_are_read_inside_their_operands(shape):
    out = _trace(*(f"mx4 {d} {' '.join(map(str, shape))}" for d in range(3)))
    assert "fno_mx4_mix_few" in out


@pytest.mark.parametrize("shape", [(1 << 22, 1, 8200, 1), (1 << 21, 6, 4100, 2), (1 << 22, 16, 1500, 1)], ids=str)
def test_millions_of_groups_of_1024_threads(shape):
    """A launch takes fewer than 2^32 threads, whatever the number of groups."""
    B, C, P, G = shape
    for d in (1, 2):
        out = _trace(f"gnorm {d} {B} {C} {P} {G} 0", f"gnorm {d} {B} {C} {P} {G} 1")
        assert "fno_gnorm_small" in out


def test_groups_that_a_team_holds():
    """The shapes of the tests of levels far from zero are held by a team, or are not, as those tests take it."""
    import test_gpu_group_norm_levels as levels
    for shapes, held in ((levels.HELD, True), (levels.SPLIT, False)):
        for B, C, P, G in shapes:
            for last in (0, 1):
                assert ("fno_gnorm_small" in _trace(f"gnorm 0 {B} {C} {P} {G} {last}")) == held, (B, C, P, G, last)
