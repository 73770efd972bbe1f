"""bench.py's output line (CPU): the totals alone, what is of single rows and kernels
goes to the standard error."""
import json

import bench


def test_the_line_is_short_and_has_what_is_needed():
    rows = {"row_%d" % i: {"ms": 1.0, "kernels_ms": {"some_kernel": 1.0}} for i in range(200)}
    needed = {"metric": bench.METRIC, "value": 1.0, "unit": "GB/s", "n_gpus": 1, "steps": 20,
              "warmup": 5, "ms_per_step": 1.0, "higher_is_better": True, "scaling": "weak",
              "vs_baseline": None, "dtype": bench.STEP_DTYPE, "data": "synthetic",
              "config": bench.job_config(1), "roofline": {}, "cpu_baseline": {}, "e2e": {},
              "gpu_launches": 1, "clocks": {}}
    line, detail = bench.split_line({**needed, "rows": rows, "kernels": rows, "extras": rows,
                                     "peaks": {}})
    assert line == needed and len(json.dumps(line)) < 2000
    assert set(detail) == {"rows", "kernels", "extras", "peaks"}
