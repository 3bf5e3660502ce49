"""The benchmark's line on stdout: whole, short, and with what its readers look for; on the CPU."""
import json

import bench


def _record(rows=12, failed=()):
    row = {"what": "decode bs=1 mr=0.5", "bs": 1, "ms_per_step": 0.7111929607391357, "parity": {"ok": True}, **{f"part_{i}_ms": 0.123456789012345 for i in range(20)}}
    decode = [{**row, "miss_rate": i / 10} for i in range(rows)]
    prefill = {"workload": "mxfp4_prefill", "tokens": 2048, "ffn_ms": 0.64, "ffn_TFLOPs": 630.0, "layer_copy_ms": 29.0,
               "overlapped_ms_per_layer": 29.5, "gate": {"rows": [0.1] * 50}, "instruction": "v_mfma"}
    configs = {f"workload_{i}": {"decode": decode, "copy_sweep": decode, "ffn": {"bs1": row}} for i in range(5)}
    configs["mxfp4_prefill"] = prefill
    return {"metric": bench.METRIC, "value": 29.29, "unit": "tok/s", "n_gpus": 1, "steps": 20, "warmup": 5, "ms_per_step": 0.711,
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
            "config": {"workload": "bf16_h2048", "bs": 1}, "tok_ms": 34.1, "copy_GBps": 57.0, "roofline": {"kernel": "copy_missing", "frac": 0.9},
            "cpu_baseline": None, "parity": {"ok": not failed, "rows_checked": 60, "failed": list(failed), "headline": {"ok": True}, "configs": {}},
            "kernels": {"expert_ffn": {"frac": 0.2, "instruction": "x"}}, "probes": {}, "decode_per_miss_rate": decode, "copy_sweep": decode,
            "configs": configs, "hybrid": {"rows": decode}, "resize": {"grow_ms": 1.0}, "prefill": prefill}


def test_the_line_is_short_and_whole():
    out = _record(failed=[("workload_0", f"row {i}") for i in range(500)])
    text = json.dumps(bench._line(out))
    assert len(text) < 8000 and "\n" not in text
    line = json.loads(text)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling", "vs_baseline", "dtype",
              "data", "config", "tok_ms", "copy_GBps", "roofline", "cpu_baseline", "probes"):
        assert line[k] == out[k], k
    assert line["parity"]["ok"] is False and line["parity"]["failed"] == [list(f) for f in out["parity"]["failed"][:20]]
    assert line["kernels"] == {"expert_ffn": {"frac": 0.2}}
    assert set(line["ms_per_step_by_workload"]) == {f"workload_{i}" for i in range(5)}
    assert len(out["configs"]) == 6 and len(out["decode_per_miss_rate"]) == 12, "the record is left as it was"


def test_an_invalid_run_says_so_in_the_line():
    out = _record()
    out["value"], out["invalid"], out["prefill"] = None, "1 measured row(s) differ", None
    line = bench._line(out)
    assert line["value"] is None and line["invalid"] == out["invalid"] and "prefill" not in line
