"""The bench's measured traffic belongs to the kernel sources that are there."""

import os
import re

import pytest

import bench
from gradient_aggregation_gb300 import workload
from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "gradient_aggregation_gb300", "csrc")


def test_hash_covers_the_device_headers_of_the_reduction():
    """fc_internal.h, the launchers' header, includes device headers too."""
    seen, todo = set(), ["fc_reduce.cu", "fc_reduce_tma.cu"]
    while todo:
        name = todo.pop()
        if name in seen or not os.path.exists(os.path.join(CSRC, name)):
            continue
        seen.add(name)
        with open(os.path.join(CSRC, name)) as f:
            todo += re.findall(r'#include "([^"]+)"', f.read())
    device = {name for name in seen if name.endswith((".cu", ".cuh"))}
    assert "fc_bulk.cuh" in device and device <= set(bench.PHASE1_SOURCES)


@pytest.mark.parametrize("name", ["alexnet", "googlenet", "nin", "stress"])
def test_profiles_are_of_the_current_kernels(name):
    """Otherwise the bench reports no traffic: take the profile again."""
    wl = workload.get(name)
    traffic = bench.traffic_from_profile(bench.kernel_source_hash(), wl)
    # every gradient is read once
    assert traffic is not None and traffic > 2 * wl.W * wl.N
