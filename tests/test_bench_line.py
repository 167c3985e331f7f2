"""The line that bench.py prints holds every field of a benchmark's result and stays short, whatever the details (no GPU needed)."""
import json
import math

import bench


def record(n):
    roof = {"bound": "mfma", "kernel": "f64_product", "what": "x" * 60, "dtype": "f64", "achieved": math.pi, "peak": 78.6,
            "unit": "TFLOP/s", "frac": 1 / 3, "flops_per_launch": 1e12, "avg_launch_ms": 1 / 7, "traffic": 1e9 / 3,
            "traffic_unit": "bytes/launch"}
    cpu = {"value": 1 / 9, "unit": "updates/s", "cores": 16, "kind": "oracle", "sample": "y" * 130, "host": {"cpu_model": "z" * 40}}
    head = {"metric": "m" * 80, "value": 1e3 / 3, "unit": "updates/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 1 / 3,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "f64+f32", "data": "synthetic",
            "config": {"workload": "w" * 30, "stacks": ["s" * 30]}, "effective_param_GBps": 1e3 / 7, "phase_ms": {f"phase{i}": 0.1 for i in range(10)},
            "phase_roofline": {f"phase{i}": roof for i in range(10)}, "eager_ms_per_step": 0.7, "roofline": roof, "qr_roofline": roof,
            "cpu_baseline": cpu}
    out = dict(head)
    out["configs"] = [dict(head, workload="w" * 30, wid=i, fp64_chain_matrices=3) for i in range(n)]
    for c in out["configs"]:
        del c["config"]
    part = {"ms_per_step": 0.2, "effective_GBps": 7e3, "bytes_per_element": 28, "roofline": roof, "cpu_baseline": cpu}
    out["elementwise"] = {"n": 1 << 26, "dtype": "f32", "data": "synthetic", "adamw": part, "lion": part}
    out["spectral"] = {"k": 32, "iters": 10, "cases": [{"workload": "g" * 30, "ms_per_call": 0.1, "roofline": roof, "cpu_baseline": cpu}] * 2}
    return out


def test_line():
    out = record(5)
    text = json.dumps(bench.line(out))
    assert len(text) < 4500
    got = json.loads(text)
    for k in ("metric", "value", "ms_per_step", "unit", "n_gpus", "steps", "warmup", "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "config"):
        assert got[k] == out[k], k
    assert [c["wid"] for c in got["configs"]] == list(range(5)) and all(c["cpu_baseline"] and c["roofline"] for c in got["configs"])
    assert got["cpu_baseline"]["kind"] == "oracle" and set(got["elementwise"]) == {"adamw", "lion"} and len(got["spectral"]) == 2


def test_line_without_the_parts():
    out = {k: v for k, v in record(0).items() if k not in ("configs", "elementwise", "spectral", "cpu_baseline")}
    assert set(bench.line(out)) == set(out) - {"phase_roofline"}
