"""The benchmark reports its verify kernel's DRAM bytes, so they have to be of the present kernel and planner sources."""
import bench


def test_traffic_is_of_the_present_sources():
    assert bench.source_fingerprint() == bench.PROFILED_FINGERPRINT
    for workload in bench.PROFILED_TRAFFIC:
        assert bench.traffic_per_launch(workload) > 0
