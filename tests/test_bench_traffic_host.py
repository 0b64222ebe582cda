"""The benchmark reports a kernel's measured HBM traffic only while the sources
that the figure was taken on are unchanged: what is beside the convolutions
stays out of those sources."""
import json
import os

import pytest

import bench
from helpers import ROOT

RECORDED = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))


@pytest.mark.parametrize("key", [k for k, v in RECORDED.items() if "source_digest" in v])
def test_recorded_traffic_belongs_to_the_sources(key):
    entry = RECORDED[key]
    assert entry["source_digest"] == bench.source_digest(entry["path"])
    assert bench.measured_traffic(key, entry["path"]) == entry["hbm_bytes_per_launch"]
