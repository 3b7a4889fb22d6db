"""The DRAM figures that the benchmark reports come from captures of the present
kernels: a record whose kernel source or shared headers changed since is not used, and
its line of the benchmark goes without."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_record_is_of_the_present_source():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        entries = json.load(f)["entries"]
    assert entries
    for e in entries:
        assert bench.traffic_for(e["kernel_src"], e["workload"]) == e["dram_bytes_per_launch"], e["workload"]
