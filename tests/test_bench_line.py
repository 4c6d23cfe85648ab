"""The length of bench.py's result line (no GPU needed)."""
import json
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402

# A configuration's entry as measure_workload makes it, every field at its full length.
FULL = {"tflops": 1234.56, "pct_of_peak": 49.06, "wall_tflops": 1234.56, "ms_per_step": 10.1234,
        "kernel_ms_mean": 10.1234, "tile": "256x256x64", "grid": 256, "k_splits": 16, "tail_tiles": 128,
        "mfma_block": 16, "clock_ghz": 2.172, "mfma_busy": 0.3898, "counter_clock_ghz": 2.3729,
        "frac_of_peak_at_counter_clock": 0.3568, "counter_mfma_busy": 0.4108, "hbm_gb_per_call": 10.2707,
        "hbm_gbps": 3497.3}


def test_result_line_fits_a_tail_of_16000_characters():
    """The headline workload's configurations in full, the other four's short;
    what else is on the line takes 3,100 characters (measured)."""
    full = {bench.label(sync, st): FULL for sync, st in bench.timed_configs(bench.HEADLINE)}
    others = {"tall32768x1024_k4096_kn%d" % i: bench.short_configs(full) for i in range(4)}
    assert set(next(iter(others.values()))) == set(full)
    head = {"M": 32768, "N": 1024, "K": 4096, "b_layout": "N x K", "best": "barrier/5", "tflops": 1234.56,
            "pct_of_peak": 49.06, "reference_tflops": 1234.56, "cpu_baseline": "x" * 330}
    line = {"modes": full, "workloads": {k: dict(head, configs=v) for k, v in others.items()}}
    assert len(json.dumps(line)) + 3500 < 16000
