"""The line that bench.py prints stays short enough to be kept whole (CPU only)."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_large_sections_stay_off_the_line():
    record = {"metric": "m", "value": 1.0, "roofline": {"bound": "hbm"}, "sweep": [1],
              "sweep_mincopy_planner": {"sweep": ["x" * 2000]}, "planners": {"mid": ["x" * 3000]},
              "other_workloads": {"mid_fwd": "x" * 9000}}
    line, details = bench.split_record(record)
    assert list(line) == ["metric", "value", "roofline", "sweep"] and all(line[k] == record[k] for k in line)
    assert {**line, **details} == record
    assert len(json.dumps(line)) < 200


def test_sections_that_were_not_measured_are_left_out():
    line, details = bench.split_record({"value": 1.0, "planners": None, "other_workloads": None})
    assert line == {"value": 1.0} and details == {}
