"""The counters that bench.py reports beside its times belong to the kernels as they are: each summary in profiles/ says of which
source files it was taken, and bench.py leaves counters of other sources out."""
import glob
import json
import os

import pytest

import bench

ROOT = os.path.dirname(os.path.abspath(bench.__file__))


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(ROOT, "profiles", "*.json"))), ids=os.path.basename)
def test_counters_are_of_the_sources_as_they_are(path):
    with open(path) as f:
        rec = json.load(f)
    assert bench.load_traffic(rec["workload"], rec["kernel"]) == rec["dram_bytes_read"] + rec["dram_bytes_write"]
