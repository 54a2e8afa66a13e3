"""The committed DRAM counters that the bench reports belong to the present sources."""

import json
import os

import bench


def test_no_entry_has_lapsed():
    # An edit of a kernel's sources, headers among them, makes the bench leave its traffic out
    # without a word. Then the launch is captured again (captured_case says how), or the
    # entry taken out.
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        kernels = json.load(f)["kernels"]
    lapsed = [k for k, e in kernels.items() if bench.traffic_for(k) != e["dram_bytes_per_full_launch"]]
    assert kernels and not lapsed, lapsed
    for k, e in kernels.items():
        assert e["dram_bytes_per_full_launch"] == e["dram_read"] + e["dram_write"], k
