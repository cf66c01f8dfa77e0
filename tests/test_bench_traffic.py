"""The measured HBM traffic that the benchmark reports comes from counter summaries of the
present grouped-GEMM sources."""
import glob
import os
import re

import pytest

import bench

FILES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "moe_gmm_*_counters.md")))
NAMES = [re.search(r"moe_gmm_(\w+)_counters", f).group(1) for f in FILES
         if "traffic_bytes_per_launch" in open(f).read()]


def test_the_default_workload_is_among_them():
    assert {"prefill", "skewed", "decode16"} <= set(NAMES)


@pytest.mark.parametrize("workload", NAMES)
def test_traffic_is_reported(workload):
    assert bench.measured_traffic(workload) > 0
