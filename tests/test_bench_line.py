"""The JSON line of bench.py's GPU arm (no GPU): short enough to be kept whole, with every key that a
reader of it needs; the whole record goes to standard error."""
import json

import bench
from hashed_head_gram_gb300 import workloads as W


def record():
    """A whole record as run_gpu collects it, with long texts and five workloads."""
    long = "a text of the record that tells how something was measured; " * 6
    roofline = {"bound": "hbm", "kernel": "project_gate_conv_and_more", "achieved": 5432.19, "peak": 6679.5, "unit": "GB/s",
                "frac": 0.8132, "bytes_per_launch": 123456789012, "basis": long, "peak_source": long,
                "achieved_no_reuse": 7432.1, "frac_no_reuse": 1.11, "frac_nominal": 0.6876, "traffic": 0.51}
    kernel = {"ms": 0.12345, "GB/s": 5432.1, "frac_hbm": 0.81, "frac_hbm_note": long, "compulsory_bytes": 1 << 40,
              "GB/s_compulsory": 4321.0, "frac_hbm_compulsory": 0.7, "roofline": roofline}
    kernels = {name: dict(kernel) for name in ("gather_sign_concat", "project_gate", "conv_residual")}
    cpu = {"value": 13033.7, "unit": "tokens/s", "cores": 16, "kind": "oracle", "threads_1": {"table": long},
           "threads_nproc": {"table": long}, "cpu_model": "a processor of some length (R) @ 2.40GHz", "sample": long}
    one = {"value": 123456789.1, "unit": "tokens/s", "steps": 100, "ms_per_step": 12.34567, "dtype": "bf16",
           "config": bench.workload_config(W.make_workload(4), 8),
           "e2e": {"value": 12345678.9, "unit": "tokens/s", "h2d_bytes_per_step": 100925440,
                   "d2h_bytes_per_step": 100663296, "how": long},
           "gpu_launches": 123456, "roofline": roofline, "kernels": kernels, "path": "two_kernel",
           "other_paths": [{"path": "fused", "ms_per_step": 1.0, "kernels": kernels}] * 3,
           "uniform_ids_control": {"ids": long, "kernels": kernels}, "rows_moved_alone": {"row_copy": {"ms": 1.0, "how": long}},
           "decode": {"steps": [{"sequences": 8, "us_per_step": 13.5}] * 4, "how": long},
           "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"], "samples": 123},
           "wall_s_timed_loop": 0.0191, "cpu_baseline": cpu}
    head = {**one, "config": bench.workload_config(W.make_workload(5), 8)}
    return {"metric": bench.METRIC, "n_gpus": 8, "warmup": 5, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "data": "synthetic: seeded Zipf token IDs, int8/64 table values, N(0,0.02) weights, N(0,1) states", **head,
            "workloads": {str(c): one for c in bench.ALL_WORKLOADS if c != 5}, "workloads_how": long}


def test_the_line_is_short_and_complete():
    rec = record()
    before = json.dumps(rec)
    line = bench.short_line(rec)
    text = json.dumps(line)
    assert len(before) > 4 * bench.LINE_BYTES and len(text.encode()) <= bench.LINE_BYTES
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
              "vs_baseline", "dtype", "data", "config", "gpu_launches", "clocks"):
        assert line[k] == rec[k], k
    assert line["e2e"] == {k: rec["e2e"][k] for k in ("value", "unit", "h2d_bytes_per_step", "d2h_bytes_per_step")}
    assert set(line["clocks"]) >= {"sm_mhz", "sm_max_mhz", "reasons"}
    assert line["roofline"]["frac"] == 0.8132 and line["kernels_ms"]["project_gate"] == 0.12345
    assert set(line["workloads"]) == {"1", "2", "3", "4"} and line["workloads"]["4"]["value"] == 123456789.1
    assert line["cpu_baseline"]["kind"] == "oracle"
    assert json.dumps(rec) == before  # the record itself stays


def test_a_line_without_extras():
    rec = record()
    for k in ("workloads", "workloads_how", "cpu_baseline"):
        del rec[k]
    line = bench.short_line(rec)
    assert "workloads" not in line and "cpu_baseline" not in line and line["value"] == rec["value"]
