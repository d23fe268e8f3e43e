"""The committed HBM counters belong to the kernels as they are: bench.py reports a
record of profiles/traffic.json only while the sources it names hash to its own
source_sha, and none of them is out of date."""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


def test_every_committed_counter_is_reported():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as fh:
        records = json.load(fh)
    assert {"dense_m16", "dense_m4096_t3"} <= set(records)
    for name, rec in records.items():
        assert bench.load_traffic(name) == rec["hbm_bytes_per_launch"], name
