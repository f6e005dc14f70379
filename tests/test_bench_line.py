"""The line that bench.py prints: the whole record's headline, short enough to survive where
only the last kilobytes of a run's output are kept (no GPU)."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def _record():
    """A record with rows as long as a run on the GPU gives them."""
    trials = {"median": 14.682, "min": 14.589, "max": 16.004, "trials": [16.004, 14.589, 14.682, 14.672, 14.896]}
    row = {"op": "w4a16", "M": 128, "K": 17408, "N": 5120, "G": 128, "kernel": "w4a16_wide_mfma_kernel",
           "launch_shape": [255, 1024, 58960], "us": 39.123, "us_trials": trials, "GBps": 3145.5, "hbm_frac": 0.3932,
           "weight_GBps": 3130.2, "TFLOPs": 601.71, "mfma_frac": 0.2243, "bytes": 46182400, "input_sha256": "8" * 64,
           "weight_copies": 28, "probe": {"same_shape": [255, 1024], "same_us": 10.093, "best_us": 8.621,
                                          "best_shape": [2048, 256], "frac_same": 0.6874, "frac_best": 0.5872}}
    stretch = lambda n: "x" * n
    return {
        "metric": bench.METRIC, "value": 2211.47, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5,
        "ms_per_step": 0.014694, "steps_timed": 20, "step_trials_ms": [0.014731] * bench.TRIALS,
        "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16", "data": "synthetic",
        "config": {"workload": stretch(120), "M": 1, "K": 5120, "N": [5120, 6144, 1024], "group_size": 128,
                   "bytes_per_step": 32495616, "input_sha256": {n: "8" * 64 for n in bench.DECODE}},
        "roofline": {"bound": "hbm", "achieved": 2824.6, "us_trials": trials, "trace": stretch(250)},
        "cpu_baseline": {"value": 1.1, "sample": stretch(300)},
        "run_record": {"device": stretch(380)},
        "chip_stream": {"best_GBps": 6222.1, "shapes": [{"shape": [209715, 1024], "us": 326.9, "GBps": 3284.3}] * 8,
                        "mfma": stretch(250)},
        "workloads": [{"workload": n, **row} for n in bench.TABLE],
        "cpu_oracle": [{"workload": n, "columns": 5120, "us": 11517.3, "GBps": 1.175, "GFLOPs": 4.552,
                        "gpu_speedup": 2037.4} for n in bench.TABLE],
        "quantizer": stretch(110), "fusion": stretch(930), "ct_ingest": stretch(60), "mxfp8_quantizer": stretch(130),
    }


def test_the_printed_line_is_short_and_whole():
    full = _record()
    text = json.dumps(bench.printed_line(full))
    assert len(json.dumps(full)) > 14000 and len(text) < 7000 and "\n" not in text
    line = json.loads(text)
    for k in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
              "vs_baseline", "dtype", "data", "config", "roofline", "cpu_baseline", "run_record"):
        assert line[k] == full[k], k
    assert line["workloads"] == {n: {"us": 39.123, "GBps": 3145.5, "TFLOPs": 601.71} for n in bench.TABLE}


def test_a_run_without_tables():
    full = dict(_record(), workloads=[], cpu_oracle=None, chip_stream=None)
    line = bench.printed_line(full)
    assert line["workloads"] == {} and line["chip_stream"] is None and line["value"] == full["value"]
    assert len(full["metric"]) and "cpu_oracle" not in line
