"""The line that bench.py prints stays short enough to be read whole, however many recipes it measures."""
import argparse
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_recipes_have_lines_of_their_own(monkeypatch, capsys):
    long = {"metric": "m" * 70, "value": 1234.56, "unit": "GB/s", "n_gpus": 1, "steps": 200, "warmup": 5, "ms_per_step": 0.1234,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "data": "synthetic", "config": {"workload": "w" * 600},
            "roofline": {"frac": 0.9248, "kernel": "k" * 300}, "e2e": {"value": 1234.56}, "cpu_baseline": {"sample": "s" * 400},
            "clocks": {"sm_mhz": 2070.0, "reasons": ["sw_power_cap"]}}
    monkeypatch.setattr(bench, "measure", lambda *a, **kw: dict(long))
    args = argparse.Namespace(workload=bench.DEFAULT_WORKLOAD, cross_mode="paged", fused=False, cpu_key_heads=9, steps=1)
    entries = bench.per_config_entries(args, 1, 0, 0, None)
    assert len(entries) == len(bench.PER_CONFIG)
    for e in entries.values():
        assert e == {"value": 1234.56, "unit": "GB/s", "ms_per_step": 0.1234, "frac": 0.9248}
    assert len(json.dumps(dict(long, per_config=entries))) < 4096
    out = capsys.readouterr()
    assert out.out == ""
    lines = [json.loads(x) for x in out.err.splitlines()]
    assert [x["per_config"] for x in lines] == list(entries) and all(x["config"] == long["config"] for x in lines)
