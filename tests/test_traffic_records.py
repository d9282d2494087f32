"""Host check (no GPU): the committed DRAM traffic records belong to the committed
kernels.  bench.py leaves a row's traffic out when a source of its kernel has changed
since the counters were taken, without a word; a change of these sources brings
records taken anew, or takes the record out."""
import json
import os
import re

import pytest

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "boolean_weight_matmul_b200", "csrc")
with open(os.path.join(ROOT, "profiles", "ncu_traffic.json")) as f:
    RECORDS = json.load(f)


def _device_headers(name):
    """The device headers (.cuh) that a source includes, directly or not."""
    with open(os.path.join(CSRC, name)) as f:
        direct = [h for h in re.findall(r'#include "(\w+\.cuh)"', f.read())]
    return set(direct).union(*[_device_headers(h) for h in direct]) if direct else set()


@pytest.mark.parametrize("key", sorted(RECORDS))
def test_traffic_record_belongs_to_the_sources(key):
    record = RECORDS[key]
    kernel = [s for s in record["sources"] if s.endswith(".cu")]
    assert len(kernel) == 1 and _device_headers(kernel[0]) <= set(record["sources"])
    assert record["source_sha256_16"] == bench.kernel_source_hash(record["sources"])
    assert bench.ncu_traffic(key) == record["dram_bytes_per_launch"] > 0
