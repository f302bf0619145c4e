"""The committed DRAM counters belong to the kernels' sources as they are."""
import json
import os

import pytest

from conftest import ROOT

bench = pytest.importorskip("bench")

with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
    TRAFFIC = json.load(f)


@pytest.mark.parametrize("key", sorted(TRAFFIC))
def test_dram_counters_are_of_these_sources(key):
    kernel, workload = key.split("|")
    assert bench.traffic_for(kernel, workload) == TRAFFIC[key]["dram_bytes_per_launch"]
    assert os.path.exists(os.path.join(ROOT, TRAFFIC[key]["summary"]))
