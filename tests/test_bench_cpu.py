"""Host-side logic of bench.py on the CPU: algorithmic work, the traffic record's
staleness rule and the reference arm's JSON line."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest

import bench
from sparse_long_context_tail_gb300 import workload as wl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_algorithmic_work_of_the_headline_workload():
    spec = wl.named_spec("llama8b-L131072")
    L, n, d, hq, hkv = 131072, spec.n_tail, spec.head_dim, spec.num_q_heads, spec.num_kv_heads
    work = bench.algorithmic_work(spec, [0, L], 1088, 2 * spec.hidden, spec.top_p)
    # query j of the tail (position L - n + j) sees L - n + j + 1 keys; two flops per multiply-add per dim
    visible = sum(L - n + j + 1 for j in range(n))
    assert work["score_pass1"]["flops"] == work["score_pass2"]["flops"] == 2.0 * d * hq * visible
    assert work["score_pass1"]["flops"] == 137372368896.0
    assert work["score_pass1"]["bytes"] == 2.0 * L * hkv * d + 2.0 * hq * d * n     # K once, tail Q once
    # gather: hidden row read and written, plus positions, slots and the index
    assert work["compact_gather"]["bytes"] == 1088 * (2.0 * 2 * spec.hidden + 32 + 4)


def test_algorithmic_work_of_requests_shorter_than_the_tail():
    spec = wl.named_spec("small-L4096")
    lengths = [1, 77, 300]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    work = bench.algorithmic_work(spec, cu, 0, 2 * spec.hidden, spec.top_p)
    visible = 0
    for L in lengths:                     # brute force: every tail query of every request
        for t in range(max(0, L - spec.n_tail), L):
            visible += t + 1
    assert work["score_pass1"]["flops"] == 2.0 * spec.head_dim * spec.num_q_heads * visible


def test_traffic_record_is_dropped_once_the_kernel_changes(tmp_path, monkeypatch):
    src = tmp_path / "sparse_long_context_tail_gb300" / "csrc"
    src.mkdir(parents=True)
    files = bench.STAGE_SOURCES["score_pass1"]
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    (tmp_path / "profiles").mkdir()
    for name in files[:-1]:
        (src / name).write_text(f"// {name} version 1\n")
    assert bench.source_sha("score_pass1") is None          # a source missing: never current
    (src / files[-1]).write_text("// header version 1\n")
    sha = bench.source_sha("score_pass1")
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(
        {"score_pass1": {"workload": "w", "source_sha": sha, "dram_bytes_per_launch": 1234}}))
    assert bench.traffic_record("score_pass1", "w") == 1234.0
    assert bench.traffic_record("score_pass1", "another workload") is None
    (src / files[-1]).write_text("// header version 2\n")   # an included header changed
    assert bench.traffic_record("score_pass1", "w") is None
    (src / files[-1]).write_text("// header version 1\n")
    assert bench.traffic_record("score_pass1", "w") == 1234.0
    (src / files[0]).write_text("// kernel version 2\n")
    assert bench.traffic_record("score_pass1", "w") is None


def test_reference_arm_prints_one_line_on_rank_zero_only():
    cmd = [sys.executable, "bench.py", "--impl", "reference", "--workload", "small-L4096", "--steps", "1",
           "--warmup", "3"]
    env = dict(os.environ, RANK="0")
    r = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stdout.splitlines() if l.startswith("{")]
    assert len(lines) == 1
    d = json.loads(lines[0])
    assert d["impl"] == "reference" and d["metric"] == bench.METRIC and d["unit"] == bench.UNIT
    assert d["value"] > 0 and d["higher_is_better"] is True and d["gpu_launches"] == 0
    assert d["cpu_baseline"]["kind"] == "oracle" and d["cpu_baseline"]["cores"] >= 1
    assert d["cpu_baseline"]["value"] == d["value"]
    assert d["e2e"] == {"value": d["value"], "unit": d["unit"], "h2d_bytes_per_step": 0, "d2h_bytes_per_step": 0}
    assert d["config"]["workload"] == "small-L4096"
    env["RANK"] = "1"
    r1 = subprocess.run(cmd, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r1.returncode == 0 and not r1.stdout.strip()


@pytest.mark.parametrize("every,layers,want", [(4, 12, [3, 7, 11]), (6, 12, [5, 11])])
def test_stack_schedules_place_the_full_attention_layers(every, layers, want):
    assert bench.full_attention_layers(layers, every) == want


def test_the_result_line_is_short_and_whole():
    """With every key of a run the line stays under 3.6 KB, and the contract's numbers are all there."""
    third = 1 / 3
    entry = {"bound": "tensor", "kernel": "score_pass1", "achieved": 1e3 * third, "peak": 1897.7, "unit": "TFLOP/s",
             "frac": third, "peak_source": "measured bf16_tflops (burst)", "traffic": None, "us_per_launch": 100 * third,
             "algorithmic_bytes_per_launch": 269484032.0, "algorithmic_flops_per_launch": 137372368896.0,
             "tflops": 1e3 * third, "gbs": 1e4 * third, "frac_of_sustained_peak": third}
    passes = {"score_pass1": entry, "score_pass2": dict(entry, kernel="score_pass2")}
    stage = {"launches": 20, "ms_per_launch": third, "share": third, "tflops": 1e3 * third, "gbs": 1e4 * third}
    stages = {n: dict(stage, launches=20 if n in ("score_pass1", "score_pass2", "select", "compact_gather") else 0)
              for n in bench.STAGES}
    spec = wl.named_spec("llama8b-L131072")

    class W:
        total_tokens = 131072

    class Args:
        gpus, no_flush = 1, False

    line = {"metric": bench.METRIC, "value": 6e8 * third, "unit": bench.UNIT, "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": third, "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic (seeded bf16 N(0,1) + planted blocks)",
            "config": bench.config_of(spec, W, Args),
            "step_ms": {k: third for k in ("median", "min", "max", "traced_mean", "stage_sum")}, "kept_tokens": 1088,
            "kept_fraction": third, "roofline": dict(entry, passes=passes), "stages": stages,
            "cpu_baseline": {"value": 1e5 * third, "unit": "tokens/s", "cores": 16, "kind": "oracle", "sample": "s" * 150},
            "e2e": {"value": 9e7 * third, "unit": "tokens/s", "h2d_bytes_per_step": 278414344, "d2h_bytes_per_step": 8946704,
                    "ms_per_step": third, "steps": 5, "serial_ms_per_step": third, "note": "n" * 450},
            "gather_p1": {k: 1e4 * third for k in ("kept_tokens", "bytes_per_launch", "gather_ms_per_launch", "achieved_gbs",
                                                   "peak_gbs", "frac", "compaction_ms_per_launch")},
            "graph": {"ms_per_step": third, "median_ms": third, "steps": 20}, "gpu_launches": 80,
            "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": [], "samples": 3}, "wall_s": third}
    text = bench.result_line(line)
    assert len(text) < 3600 and "\n" not in text
    got = json.loads(text)
    assert set(got) == set(line)
    for k in ("metric", "unit", "n_gpus", "steps", "warmup", "higher_is_better", "scaling", "dtype", "data", "config",
              "gpu_launches", "clocks", "vs_baseline"):
        assert got[k] == line[k]
    assert got["value"] == pytest.approx(line["value"], rel=1e-6) and got["e2e"]["h2d_bytes_per_step"] == 278414344
    assert got["roofline"]["algorithmic_flops_per_launch"] == 137372368896
    assert list(got["stages"]) == ["score_pass1", "score_pass2", "select", "compact_gather"]
    assert list(got["roofline"]["passes"]) == ["score_pass2"]
