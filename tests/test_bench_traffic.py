"""The benchmark reports the GEMM's measured DRAM traffic only where it was taken on the sources that are there."""
import bench


def test_traffic_was_measured_on_these_sources():
    assert bench.committed_traffic(), "profiles/gemm_traffic.json is of other GEMM sources: capture it again"
