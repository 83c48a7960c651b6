"""The committed traffic counters belong to the GEMM's present sources, so
bench.py reports measured HBM bytes (no GPU)."""
import os

import pytest

import bench


@pytest.mark.parametrize("workload", ["dsv3_skew", "mixtral"])
def test_the_committed_counters_are_valid(workload):
    assert os.path.exists(bench.traffic_file(workload))
    assert bench.measured_traffic(workload) > 1e9
