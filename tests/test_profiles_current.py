"""The recorded DRAM traffic (profiles/traffic.json) belongs to the kernels as they are: the bench reports an entry only
while its hash is that of the kernel's source, so a change of the source without a new capture loses the figure."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

SOURCES = {"power-law": ("spx_spmv.cu", "spx_gather.cuh", "spx_carveout.cuh"), "dual": ("spx_spmv.cu", "spx_gather.cuh", "spx_carveout.cuh"),
           "power-law-coo": ("spx_coo.cu", "spx_gather.cuh", "spx_carveout.cuh"),
           "power-law-sell": ("spx_sell.cu", "spx_gather.cuh", "spx_carveout.cuh"),
           "wcsr": ("spx_wcsr.cu", "spx_tc.cuh"), "wcsr-skewed": ("spx_wcsr.cu", "spx_tc.cuh"),
           "bsr": ("spx_bsr.cu", "spx_tc.cuh"), "bsr-skewed": ("spx_bsr.cu", "spx_tc.cuh")}
TRAFFIC = json.load(open(os.path.join(ROOT, "profiles", "traffic.json")))


@pytest.mark.parametrize("workload", sorted(TRAFFIC))
def test_recorded_traffic_is_of_the_present_source(workload):
    files = SOURCES.get(workload, ("spx_spmm.cu",))
    assert bench.traffic_from_profile(workload, bench.source_hash(*files)) == TRAFFIC[workload]["dram_bytes_per_launch"]
