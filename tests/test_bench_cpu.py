"""bench.py's reference arm (the CPU oracle) runs without a GPU: check its
JSON line carries the contract's keys."""
import json
import os
import subprocess
import sys

from conftest import ROOT


def test_reference_arm_prints_one_contract_line():
    res = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--impl", "reference",
                          "--steps", "2", "--warmup", "3"], capture_output=True, text=True,
                         timeout=600, cwd=ROOT)
    assert res.returncode == 0, res.stderr
    lines = [l for l in res.stdout.splitlines() if l.strip()]
    assert len(lines) == 1
    d = json.loads(lines[0])
    for key in ("impl", "metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step",
                "higher_is_better", "scaling", "vs_baseline", "dtype", "data", "config",
                "cpu_baseline", "e2e"):
        assert key in d, key
    assert d["impl"] == "reference" and d["value"] > 0 and d["steps"] == 2
    assert d["cpu_baseline"]["kind"] == "oracle"
    assert d["cpu_baseline"]["cores"] == len(os.sched_getaffinity(0))   # every host core
    assert d["e2e"]["h2d_bytes_per_step"] == 0 and d["e2e"]["d2h_bytes_per_step"] == 0


def test_warmup_below_three_is_refused():
    res = subprocess.run([sys.executable, os.path.join(ROOT, "bench.py"), "--impl", "reference",
                          "--steps", "1", "--warmup", "2"], capture_output=True, text=True,
                         timeout=300, cwd=ROOT)
    assert res.returncode != 0


def test_every_mode_has_its_function():
    import bench
    for name in ("bench_gpu", "bench_e2e", "bench_only", "bench_configs", "bench_sweep",
                 "bench_reference", "cpu_baseline", "aggregate_gbs"):
        assert callable(getattr(bench, name, None)), name


def test_link_bound_closed_forms():
    """The e2e step's link bound: with no device-to-host bytes it is the
    host-to-device time alone; with a link whose directions do not slow each
    other it is the longer direction's time; with equal bytes both ways it is
    the time of both at their shared rates."""
    import bench

    free = {"h2d_gbs": 200.0, "d2h_gbs": 100.0, "both": {"h2d_gbs": 200.0, "d2h_gbs": 100.0}}
    assert abs(bench.link_bound_gbs(10**9, 0, 10**9, free) - 200.0) < 1e-9
    assert abs(bench.link_bound_gbs(10**9, 10**9, 2 * 10**9, free) - 200.0) < 1e-9   # 10 ms
    shared = {"h2d_gbs": 210.0, "d2h_gbs": 190.0, "both": {"h2d_gbs": 170.0, "d2h_gbs": 170.0}}
    assert abs(bench.link_bound_gbs(17 * 10**8, 17 * 10**8, 34 * 10**8, shared) - 340.0) < 1e-6
    # 1.7 GB in, 0.85 GB out: 5 ms both ways, then 0.85 GB in alone at 210 GB/s
    t = 0.005 + 0.85e9 / 210e9
    assert abs(bench.link_bound_gbs(17 * 10**8, 85 * 10**7, 10**9, shared) - 1.0 / t) < 1e-6


def test_default_line_is_short_and_whole():
    """Everything a reader of the line needs, in 1500 characters, whatever the record holds."""
    import bench

    kernel = {"ms": 0.1585, "bytes": 1 << 30, "gbs": 6776.4, "ms_host_launched": 0.1591, "stages": 3, "tile": [128, 64]}
    full = {"metric": "achieved HBM GB/s (read+write) for pipelined tile copy + rowsum", "value": 6811.2, "unit": "GB/s",
            "n_gpus": 8, "steps": 2000, "warmup": 5, "ms_per_step": 0.3153, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": "f16 copy + bf16->f32 rowsum", "data": "synthetic (seeded, drawn on device)",
            "config": {"workload": "tile_copy fp16 16384x16384 tile 128x64 + tile_rowsum bf16 8192x65536 tile 64x256",
                       "copy_stages": 3, "rowsum_stages": 2, "streams": "x" * 200, "launch": "x" * 200,
                       "l2": "inputs (512 MiB, 1 GiB) larger than L2; no flush",
                       "parallelism": "independent replica per GPU x8"},
            "frac_of_peak": 1.003, "value_one_stream": 6726.1, "value_host_launched": 6825.3,
            "kernels": {"copy": kernel, "rowsum": kernel},
            "roofline": {"bound": "hbm", "kernel": "mbt_rowsum_kernel", "achieved": 6776.4, "peak": 6790.3, "unit": "GB/s",
                         "frac": 0.998, "traffic": 1076517120, "timing": "x" * 800},
            "e2e": {"value": 251.2, "unit": "GB/s", "h2d_bytes_per_step": 1610612736, "d2h_bytes_per_step": 536903680,
                    "link": {"h2d_gbs": 210.0}, "link_bound": 258.9, "link_note": "x" * 400},
            "gpu_launches": 4000, "sweep": [{"x": "y" * 400}] * 30, "flat_points": [{"x": "y" * 400}] * 5,
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "power_w_max": 906.06, "samples": 120,
                       "reasons": ["sw_power_cap"]},
            "cpu_baseline": {"value": 19.5651, "unit": "GB/s", "cores": 16, "kind": "oracle", "sample": "x" * 400}}
    line = bench.headline(full)
    text = json.dumps(line)
    assert len(text) <= 1500, len(text)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "e2e", "gpu_launches", "clocks", "roofline", "cpu_baseline"):
        assert key in line, key
    assert line["value"] == 6811.2 and line["clocks"]["reasons"] == ["sw_power_cap"]
    assert line["e2e"] == {"value": 251.2, "unit": "GB/s", "h2d_bytes_per_step": 1610612736,
                           "d2h_bytes_per_step": 536903680, "link_bound": 258.9}
