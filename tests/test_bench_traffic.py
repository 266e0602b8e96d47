"""The bench's traffic figures are those of the kernels as they are: profiles/traffic.json holds
them with a hash of the sources that were captured, and the bench drops a figure whose sources
have changed.  Runs without a GPU."""
import json
import os

import pytest

import bench

SOURCES = {"fwd": "fwd_tc.cuh", "dkdv": "bwd_tc.cuh", "dq": "bwd_tc.cuh"}


@pytest.mark.parametrize("kernel", sorted(SOURCES))
def test_traffic_figures_belong_to_the_sources(kernel):
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        want = json.load(f)[kernel]["bytes_per_launch"]
    assert bench.traffic_for(kernel, bench.src_sha(SOURCES[kernel], "common.cuh")) == want
