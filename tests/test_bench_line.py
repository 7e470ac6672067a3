"""The line that bench.py prints: the fields of its contract, and short enough to be found whole at the end of a log."""
from __future__ import annotations

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

LIMIT = 8000  # characters


def launch(patterns):
    e = {"us": 12.345, "p10": 12.345, "p90": 12.345, "launches": 12345, "GBs": 1234.5, "pct_peak": 77.7, "rotation_MB": 1234,
         "speedup_vs_dense": 1.234, "speedup_vs_hipblaslt": 1.234, "speedup_vs_best_dense": 1.234}
    d = {p: dict(e) for p in patterns}
    return {"R": [14336, 14336], "K": 14336, **d, "dense_us": 1.5, "dense_GBs": 1.5, "hipblaslt_us": 1.5,
            "stream_read": {"us": 1.5, "GBs": 1.5, "pct_peak": 70.1}}


def full():
    labels = ["q", "k", "v", "o", "gate", "up", "down", "q|k|v", "gate|up+swiglu"]
    step = {"launches": 256, "ms": 0.1234, "GBs": 5432.1, "pct_hbm_peak": 65.4, "dense_ms": 1.2345, "speedup_vs_dense": 2.345,
            "launch_sum_vs_best_dense": {"sparse_us": 1.2, "dense_us": 1.2, "speedup": 1.9}}
    configs = {}
    for name, layers, batches in bench.OTHER_CONFIGS:
        patterns = [f"{n}:{m}" for n, m in bench.CONFIGS[name]["patterns"]]
        configs[name] = {"workload": bench.CONFIGS[name]["workload"], "layers": layers, "patterns": patterns, "seconds": 9.9,
                         "by_batch": {f"B{b}": {"step": dict(step), "per_layer": {x: launch(patterns) for x in labels}}
                                      for b in batches}}
    per = {x: launch(["2:4", "16:32"]) for x in labels}
    check = {f"{x} {p}": {"pct_peak": 70.0, "speedup_vs_dense": 1.5, "pct_ok": x != "k", "speedup_ok": True}
             for x in labels for p in ("2:4", "16:32")}
    return {"metric": bench.METRIC, "value": 5123.3, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 0.7666,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
            "config": {"workload": bench.CONFIGS["8b"]["workload"], "layers": 8, "batch": 1, "patterns": ["2:4", "16:32"],
                       "parallelism": "single GPU"},
            "pct_hbm_peak": 65.0, "step": dict(step, groups=labels), "unfused_step": dict(step), "per_layer": per,
            "per_layer_target": {"criterion": "c" * 100, "launches": check}, "configs": configs,
            "metadata_formats": {x: launch(["2:4"]) for x in labels}, "unstructured_50": {x: launch(["2:4"]) for x in labels},
            "solver": launch(["2:4"]), "pack_GBs": 1.5, "parity": "ok",
            "roofline": {"bound": "hbm", "achieved": 5863.2, "peak": 8000.0, "kernel": "k" * 80},
            "cpu_baseline": {"value": 3.9, "sample": "s" * 100, "one_core": {"value": 1, "sample": "s" * 60}}}


def test_the_line_is_short_and_has_the_contract_s_fields():
    out = full()
    line = json.dumps(bench.headline(out))
    assert len(json.dumps(out)) > 2 * LIMIT  # what it is taken from is not
    assert len(line) < LIMIT, len(line)
    got = json.loads(line)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline",
              "dtype", "data", "config", "roofline", "cpu_baseline"):
        assert got[k] == out[k], k
    assert got["per_layer"]["gate"]["2:4"] == [12.345, 77.7, 1.234]
    assert got["per_layer_target"]["launches"] == 18 and got["per_layer_target"]["met"] == 16
    assert got["configs"]["70b"]["B4"]["pct_hbm_peak"] == 65.4


def test_a_run_without_the_other_workloads():
    out = dict(full(), configs=None, metadata_formats=None, unstructured_50=None, solver=None)
    assert bench.headline(out)["configs"] is None
