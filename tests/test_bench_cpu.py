"""bench.py without a GPU."""
import bench
import pytest


@pytest.mark.parametrize("workload", sorted(bench.HBM_COUNTERS))
def test_recorded_traffic_belongs_to_the_current_sources(workload):
    """A change to the expert GEMMs' sources needs its HBM counters taken again;
    until then the bench reports no traffic."""
    assert bench.counted_traffic(workload) is not None
