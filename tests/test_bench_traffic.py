"""The recorded memory traffic that the benchmark reports belongs to the kernel
sources as they are (CPU): a source that changes without a new capture loses the
figure."""
import os

import pytest

import bench


@pytest.mark.parametrize("path", bench.TRAFFIC_FILES, ids=os.path.basename)
def test_recorded_traffic_is_of_the_present_sources(path):
    v = bench.read_traffic_file(path)
    assert v["source_sha256"] == bench.sources_sha(v["sources"].split())
    assert bench.recorded_traffic(int(v["workload"]), int(v["layers"]), v["verify"]) == int(v["dram_bytes_per_launch"])
