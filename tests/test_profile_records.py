"""The recorded DRAM traffic of the prompt kernels belongs to their present sources: a change of a kernel, or of a header it
is built from, needs a new capture (or its record taken out), or the benchmark has no traffic to report."""
import json

import pytest

import bench


@pytest.mark.parametrize("workload,source", [("wide_beam_b128_w96", "bsp_wide.cu"), ("qwen3_0p6b_b64_w30", "bsp_prefix.cu")])
def test_traffic_record_matches_the_sources(workload, source):
    with open(bench.PROFILE_TRAFFIC) as f:
        records = [r for r in json.load(f)["records"] if r["workload"] == workload]
    for r in records:
        assert r["kernel_source_sha"] == bench.kernel_source_hash(source)
        assert bench.profiled_traffic(workload, r["kernel"].split("<")[0], source) == r["dram_bytes_per_launch"]
