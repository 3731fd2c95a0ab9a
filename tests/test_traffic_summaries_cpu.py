"""The committed counter summaries belong to the sources as they are: where a source that one
of them names has changed, the benchmark reports no traffic for that kernel."""

import glob
import os
import re

import pytest

import bench

FILES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*_traffic.md")))
NAMED = [f for f in FILES if re.search(r"^traffic_bytes_per_launch:", open(f).read(), re.M)]


@pytest.mark.parametrize("path", NAMED, ids=os.path.basename)
def test_summary_is_current(path):
    kernel, cfg, dtype = re.fullmatch(r"(\w+)_(c\d)_(\w+)_traffic\.md", os.path.basename(path)).groups()
    assert bench.measured_traffic(kernel, cfg, dtype) > 0


def test_every_headline_workload_has_its_traffic():
    have = {re.fullmatch(r"\w+?_(c\d_\w+)_traffic\.md", os.path.basename(f)).group(1) for f in NAMED}
    assert {f"{name}_{dt}" for name, dt in bench.METRIC_CONFIGS} <= have
