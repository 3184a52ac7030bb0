"""The DRAM traffic that the bench line reports comes from captures of the sources as they are."""
import os

import pytest

import bench

LINES = [line.split() for line in open(os.path.join(bench.ROOT, "profiles", "traffic.txt"))
         if line.strip() and not line.startswith("#")]


@pytest.mark.parametrize("kernel,workload,moved,sha", LINES, ids=lambda v: str(v))
def test_recorded_traffic_is_of_these_sources(kernel, workload, moved, sha):
    assert bench.kernel_source_sha(kernel) == sha
    assert bench.recorded_traffic(kernel, workload) == float(moved)
