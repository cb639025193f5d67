"""The DRAM-traffic records that bench.py reports belong to the kernels as they
are: a record of an older source is taken again or removed (no GPU)."""
from __future__ import annotations

import json
import os

import bench


def test_every_record_is_of_the_present_source():
    with open(os.path.join(bench.ROOT, "profiles", "ncu_traffic.json")) as f:
        records = json.load(f)
    for workload, r in records.items():
        got = bench.ncu_traffic(workload, r["source"])
        assert got == r["dram_bytes_read"] + r["dram_bytes_write"], workload
        assert os.path.exists(os.path.join(bench.ROOT, r["summary"].split(" ")[0]))
