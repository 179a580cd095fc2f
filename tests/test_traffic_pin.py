"""The committed traffic measurements (profiles/traffic.json) belong to the
committed kernel sources: an entry whose source files changed since is silently
left out of the benchmark's roofline, so a change to them comes with a new
measurement (no GPU needed to notice)."""
import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_measurements_match_their_sources():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        entries = json.load(f)
    assert entries
    for name, e in entries.items():
        assert bench.src_hash(e["src_files"]) == e["src_hash"], f"{name}: taken on another state of {e['src_files']}"


def test_benchmark_reports_the_traffic_of_its_default_workload():
    assert bench.traffic_for("C2", 16) == 451657728
