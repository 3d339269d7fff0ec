"""The counter summaries that the bench reads were taken on the scan kernels as
they are: helpers of other operators stay out of the scan's sources."""
import bench


def test_traffic_summaries_are_of_these_kernels():
    sha = bench.kernel_source_sha()
    assert bench.load_traffic(sha) is not None
    assert bench.load_decode_ratio(sha) is not None
