"""The line bench.py prints: every field of its contract, short enough to be read
whole from the end of a captured output."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402
from newton_schulz_bucket_gb300 import workloads as W  # noqa: E402


def _record():
    f = 1234567.890123456
    steps = {"median": f, "min": f, "max": f}
    clocks = {"sm_mhz": 1447.0, "sm_max_mhz": 2070.0, "samples": 1000,
              "reasons": ["sw_power_cap", "hw_thermal_slowdown", "sw_thermal_slowdown"]}
    peaks = {"hbm_gbs": f, "bf16_tflops_sustained": f, "source": "measured"}
    group = {"shape": [16384, 16384], "batch": 1000, "path": "tensor", "bound": "tensor", "ms": f, "TFLOP_s": f,
             "roofline_frac": f, "executed_flop_fraction": f, "TFLOP_s_executed": f, "roofline_frac_executed": f}
    oracle = {"value": f, "unit": "TFLOP/s", "cores": 16, "host_cores": 16, "blas": "scipy-openblas 0.3.34.106.0",
              "kind": "oracle", "sample": "x" * 260, "ms_per_step": f, "wall_s": f}
    entries = []
    for name, k in bench.PER_CONFIG:
        w = W.get(name, k)
        entries.append({"workload": w.name, "shapes": bench.describe_shapes(w.shapes), "ns_steps": w.ns_steps, "value": f,
                        "unit": "TFLOP/s", "ms_per_step": f, "step_ms_this_rank": steps, "matrices_per_s": f,
                        "tflops": f, "gbs": f, "tflops_executed": f, "per_group": [group] * 12,
                        "roofline": bench.roofline_of(w, group, peaks), "clocks": clocks, "cpu_baseline": oracle})
    w = W.get(bench.DEFAULT_CONFIG)
    return {"metric": bench.METRIC, "value": f, "unit": "TFLOP/s", "n_gpus": 8, "steps": 1000, "warmup": 100,
            "ms_per_step": f, "step_ms_this_rank": steps, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic: seeded Gaussian G, M0, P (per-config stds); no dataset",
            "config": bench.config_dict(w, 8), "matrices_per_s": f, "tflops": f, "gbs": f, "tflops_executed": f,
            "per_group": [group] * 4, "roofline": bench.roofline_of(w, group, peaks), "cpu_baseline": oracle,
            "e2e": {"value": f, "unit": "TFLOP/s", "ms_per_step": f, "steps": 6, "step_ms_this_rank": steps,
                    "h2d_bytes_per_step": 10 ** 11, "d2h_bytes_per_step": 10 ** 11},
            "gpu_launches": 100000, "clocks": clocks, "wall_s_timed": f, "per_config": entries}


def test_the_line_is_short_and_whole():
    record = _record()
    line = bench.result_line(record)
    assert "\n" not in line and len(line) < 2500, len(line)
    d = json.loads(line)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "gpu_launches", "roofline", "cpu_baseline", "clocks", "e2e"):
        assert key in d, key
    assert d["config"] == bench.rounded(record["config"]) and d["e2e"].keys() == record["e2e"].keys()
    assert abs(d["value"] / record["value"] - 1) < 1e-5
    assert len(d["per_config"]) == len(bench.PER_CONFIG)
    assert len(json.dumps(record)) > 3000  # what was printed before: longer than the 3000 characters a reader kept


def test_a_line_without_the_optional_parts():
    record = _record()
    record.update(per_config=None, cpu_baseline=None, e2e=None)
    d = json.loads(bench.result_line(record))
    assert "per_config" not in d and d["e2e"] is None and d["cpu_baseline"] is None
