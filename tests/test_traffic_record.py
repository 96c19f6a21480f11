"""The DRAM bytes that the bench reports beside its roofline are counters of the
present kernels: profiles/traffic.json names the sources they were taken with."""
import json
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORD = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))


@pytest.mark.parametrize("key", sorted(RECORD))
def test_counters_are_of_the_present_sources(key):
    assert bench._profiled_traffic(key) == RECORD[key]["dram_bytes_per_launch"]
    assert os.path.exists(os.path.join(ROOT, RECORD[key]["profile"]))
