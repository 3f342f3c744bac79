"""The committed traffic records are of the present kernel sources: bench.py leaves out a record of any
other source, so an edit of a profiled file has to come with a new capture."""

import hashlib
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RECORDS = json.load(open(os.path.join(ROOT, "profiles", "ncu_traffic.txt")))


@pytest.mark.parametrize("key", [k for k, v in RECORDS.items() if isinstance(v, dict)])
def test_record_and_summary_are_of_the_present_source(key):
    rec = RECORDS[key]
    with open(os.path.join(ROOT, rec["source"]), "rb") as f:
        sha = hashlib.sha256(f.read()).hexdigest()
    assert rec["sha256"] == sha
    with open(os.path.join(ROOT, rec["capture"])) as f:
        assert sha[:8] in f.read()


def test_bench_reports_both_records():
    import sys

    sys.path.insert(0, ROOT)
    import bench

    assert set(bench.load_traffic()) == {"decode", "prefill"}
