"""CPU test of the benchmark's line: short enough to be read whole from the output's end."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_other_workloads_are_short_and_keep_their_main_figures():
    stats = {k: 23.070400208234787 for k in ("mean", "median", "p10", "p90", "min", "max", "n")}
    r = {"workload": "x" * 170, "batch": 256, "context_tokens": 407706, "num_splits": 11,
         "splits": {"mode": "plan", "records": 11}, "decode_us": 23.070400208234787, "decode_us_stats": stats,
         "decode_gbs": 3645.992060856232, "decode_frac": 0.545146164210498, "stream_read_frac_same_bytes": 0.656132081690085,
         "layered": {"frac": 0.6919421098796217, "gbs": 1.0}, "step": {"tokens_per_s": 1215214.4983804633, "chained_us": stats},
         "cache_fill": {"gbs": 4895.068618196236, "hbm_frac": 0.7319072110459226, "us_stats": stats},
         "e2e": {"value": 1073940.818521542, "step_us": stats}, "cpu_baseline": {"value": 50.91102375073552, "sample": "y" * 300},
         "cpu_baseline_all_cores": {"value": 807.053705982191, "sample": "y" * 300}, "err_flag": 0}
    f = bench.main_figures(r)
    assert f["decode_us"] == 23.0704 and f["decode_frac"] == 0.545146 and f["err_flag"] == 0 and f["step_us"] == 23.0704
    assert f["e2e_tokens_per_s"] == 1073940.0 and f["cpu_tokens_per_s"] == 50.911 and f["layered_frac"] == 0.691942
    assert len(json.dumps(f)) < 600
    # parts that a run leaves out are left out here too
    assert bench.main_figures({"batch": 1, "e2e": None, "cpu_baseline_all_cores": None}) == {"batch": 1}
