"""The bench reports the main kernel's DRAM traffic only from a capture of the sources that
it runs: the headline workload has one."""
import bench


def test_the_headline_workload_has_a_record_of_these_sources():
    src = bench.kernel_source_hash(bench.MAIN_KERNEL_SOURCES["tc"])
    bytes_per_launch = bench.recorded_traffic("bumps3_512cubed_r2000", "tc", src)
    # two fp16 images of 512^3 values at least once
    assert bytes_per_launch is not None and bytes_per_launch >= 2 * 2 * 512 ** 3
