"""The line bench.py prints: whole within the last 3000 characters of stdout,
whatever the other workloads' entries hold."""
import json

import bench


def entry(name, metric="paged decode KV GB/s"):
    """An entry as long as the measured ones."""
    x = 123456.78901234567
    return {"metric": metric, "value": x, "unit": "GB/s", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": x / 1e6, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic", "config": {"workload": name, "text": "c" * 280}, "queries_per_s": x,
            "roofline": {"bound": "hbm", "achieved": x, "peak": 6693.8, "unit": "GB/s", "frac": 0.892062697654423,
                         "traffic": 1122624256.0, "kernel": "k" * 160, "work_per_launch": 1111013312,
                         "avg_launch_ms": 0.1860592007637024, "peak_source": "measured hbm_gbs"},
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": [], "samples": 8, "window": "w" * 70},
            "e2e": {"value": x, "unit": "GB/s", "h2d_bytes_per_step": 851712, "d2h_bytes_per_step": 532480,
                    "steps": 50, "loop": "l" * 330}, "gpu_launches": 60,
            "aux": {"scatter": {"ms": x / 1e9, "bytes": 524800, "GB/s": x, "timing": "20 calls in one CUDA graph replay"}},
            "cpu_baseline": {"value": x, "unit": "GB/s", "cores": 16, "host_cores": 16, "kind": "oracle",
                             "sample": "s" * 130, "one_thread": {"value": x, "unit": "GB/s", "cores": 1,
                                                                 "sample": "t" * 100}}}


def test_one_short_line(capsys):
    names = list(bench.EXTRA_WORKLOADS)
    extra = {n: entry(n) for n in names}
    line = entry("gqa_decode")
    bench.report(line, extra)
    got = capsys.readouterr()
    assert got.out.count("\n") == 1 and len(got.out) < 3000
    d = json.loads(got.out)
    assert {k: d[k] for k in ("metric", "unit", "steps", "config")} == {k: line[k] for k in ("metric", "unit", "steps", "config")}
    for k in ("value", "ms_per_step"):  # seven digits
        assert abs(d[k] - line[k]) <= 1e-6 * line[k]
    assert d["e2e"]["h2d_bytes_per_step"] == 851712 and d["gpu_launches"] == 60
    assert list(d["workloads"]) == names
    assert all(v == [123460.0, "GB/s", 0.1235, 0.892] for v in d["workloads"].values())
    assert json.loads(got.err)["workloads"] == extra and "workloads" not in line


def test_one_workload_alone(capsys):
    bench.report(entry("tiny_decode"), {})
    got = capsys.readouterr()
    assert "workloads" not in json.loads(got.out) and got.err == ""
