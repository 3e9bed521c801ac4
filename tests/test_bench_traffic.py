"""bench.py's measured bytes (CPU): each was taken with the kernels as they are, so that none is reported as unknown."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("bench_traffic", os.path.join(ROOT, "bench.py"))
bench = importlib.util.module_from_spec(spec)
spec.loader.exec_module(bench)


@pytest.mark.parametrize("workload,kernel", sorted(bench.MEASURED_TRAFFIC))
def test_measured_traffic_is_of_these_kernels(workload, kernel):
    assert bench.traffic_of(workload, kernel) == bench.MEASURED_TRAFFIC[workload, kernel][2]
