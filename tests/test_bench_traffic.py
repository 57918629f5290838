"""The DRAM figures that bench.py reports are recorded captures, each tied to the
sources of its kernel by their hash; a capture of other sources is reported as null.
A change to those sources needs a new capture (or its entry taken out)."""
import json
import os

import pytest

import bench

PATH = os.path.join(bench.ROOT, "profiles", "dram_traffic.json")
with open(PATH) as f:
    RECORDED = json.load(f)


@pytest.mark.parametrize("kernel,workload", [(k, w) for k, v in RECORDED.items() for w in v])
def test_recorded_traffic_is_of_these_sources(kernel, workload):
    assert bench.recorded_traffic(kernel, workload) == RECORDED[kernel][workload]["dram_bytes_per_launch"]


def test_the_headline_kernel_has_one():
    assert bench.recorded_traffic(bench.HEADLINE_KERNEL, "nt_projection")
