"""Host logic of bench.py's line (no GPU): with several workloads it stays
short enough to be read whole, and keeps the headline's contract keys."""
import importlib.util
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(monkeypatch):
    spec = importlib.util.spec_from_file_location("bench_line_under_test", os.path.join(ROOT, "bench.py"))
    mod = importlib.util.module_from_spec(spec)
    monkeypatch.setattr(sys, "argv", ["bench.py"])
    spec.loader.exec_module(mod)
    return mod


def entry(v):
    """An entry of the size that a run's have: about 5.7 KB."""
    note, x = "how this number was taken, in a sentence or two " * 3, v / 3
    timed = dict(ms_per_step=x, tokens_per_s=x, hbm_frac=x, note=note)
    kernels = dict(route=x, dispatch=x, combine=x)
    return dict(
        metric="m", value=v, unit="tokens/s", n_gpus=1, steps=20, warmup=5, ms_per_step=x, higher_is_better=True,
        scaling="weak", vs_baseline=None, dtype="bf16", data=note, config=dict(workload="w", l2=note), hbm_gbs=x,
        hbm_frac=x, R=5, roofline=dict(bound="hbm", kernel="combine", achieved=x, frac=x, timing=note, other=note),
        kernels_ms=kernels, kernels_gbs=kernels, execution=note, unpipelined=timed, pipelined=timed, graph=timed,
        gpu_launches=60, clocks=dict(sm_mhz=2070.0, sm_max_mhz=2070.0, reasons=[], note=note),
        combine_ulp=dict(beyond_1ulp=3, outside_bound=0, note=note),
        e2e=dict(value=x, unit="tokens/s", h2d_bytes_per_step=8, d2h_bytes_per_step=16, path=note),
        cpu_baseline=dict(value=x, cores=1, sample=note, threaded=dict(sample=note)),
        backward=dict(ms_per_pass=x, kernels_ms=kernels, kernels_frac=kernels, algorithmic_bytes=kernels, note=note * 3),
        dedup=dict(send_over_packed=x, dispatch_frac=x, by_ranks={str(i): kernels for i in range(8)}, note=note * 3))


def test_the_line_of_all_workloads_is_short(monkeypatch):
    bench = load(monkeypatch)
    entries = {n: entry(1e8 * (i + 1)) for i, n in enumerate(bench.DEFAULT_WORKLOADS)}
    line = bench.contract_line(entries, bench.HEADLINE_WORKLOAD)
    assert len(json.dumps(line)) < 8000 < len(json.dumps(entries))
    head = entries[bench.HEADLINE_WORKLOAD]
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "roofline", "cpu_baseline", "clocks", "e2e", "gpu_launches"):
        assert line[key] == head[key], key
    assert set(line["workloads"]) == set(entries)
    for n, e in line["workloads"].items():
        assert e["hbm_frac"] == float(f"{entries[n]['hbm_frac']:.5g}") and set(e["graph"]) == {"ms_per_step", "hbm_frac"}
    # one workload: its whole entry
    assert bench.contract_line({"tiny": head}, "tiny") == head
