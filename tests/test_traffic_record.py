"""The DRAM traffic that bench.py reports belongs to the kernels as they are."""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "dram_traffic.json")) as f:
    KEYS = sorted(k for k in json.load(f) if not k.startswith("_"))


@pytest.mark.parametrize("key", KEYS)
def test_sources_are_those_of_the_capture(key):
    """(A changed source needs a new capture, or the figure is left out.)"""
    assert bench.traffic_for(key) is not None
