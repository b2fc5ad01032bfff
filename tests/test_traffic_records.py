"""The committed counter records belong to the committed kernels, so bench.py reports their HBM traffic (it gives null
for a record of other sources, shared headers included)."""
import json

import pytest

import bench


@pytest.mark.parametrize("config", sorted(bench.TRAFFIC))
def test_traffic_record_is_of_these_sources(config):
    rec = json.load(open(bench.traffic_file(config)))
    assert rec["source_sha"] == bench.gemm_source_sha(config), "take the counters again"
    assert bench.traffic_bytes(config) == rec["bytes_per_step"] > 0
