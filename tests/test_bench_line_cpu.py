"""bench.py's printed line: the contract's keys and every configuration's
times, short enough for the tail of a log to hold it whole (no GPU)."""
import json


def _record(bench):
    q = {"median": 10.872650146484375, "p10": 10.804250165820122, "p90": 10.932800024747849, "mean": 10.876127444207668}
    k = {"us": q, "bound": "hbm", "achieved": 403.9337656303243, "peak": 8000.0, "unit": "GB/s", "frac": 0.05049172070379054,
         "algorithmic_bytes": 1573120.0}
    mode = {"us_per_call": q, "effective_TOPS": 197.51243892404463, "kernels": {"quantize": k, "gemm": k}}
    configs = [{"id": c[0], "workload": c[1], "shape": "4096x5120x5120", "fmt": "nvfp4", "warm": mode, "cold": mode,
                "vendor_gemm": {"kind": "bf16 torch.matmul", "us": 137.97255158424377, "TOPS": 1556.4571527756243}}
               for c in bench.CONFIGS]
    del configs[0]["cold"]
    nexts = [dict(configs[1], id=c[0], row=c[2]) for c in bench.NEXT]
    roof = dict(k, kernel="w8a8_linear int8 64x2048x8192 (gemm_int_decode_kernel)", timing="x" * 90, us=6.1,
                frac_of_measured_copy=0.5, warm=dict(k), traffic=17572096.0,
                profile={"median_us": 6.0, "mean_us": 6.1, "frac": 0.3, "source": "profiles/bench_kernels.txt [C2b cold gemm]"})
    cpu = {"value": 0.07, "unit": "TOPS", "cores": 16, "kind": "oracle", "sample": "y" * 400, "single_thread_value": 0.01,
           "host_cores": 128, "cpu_model": "AMD EPYC 9575F 64-Core Processor", "configs": {c[0]: {"single": q, "all": q} for c in bench.CONFIGS}}
    return {"metric": bench.METRIC, "value": 154.78921721542116, "unit": "TOPS", "n_gpus": 1, "steps": 20, "warmup": 5,
            "ms_per_step": 0.01734, "us_per_call": q, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
            "dtype": "i8", "data": "synthetic (seeded)", "config": {"workload": bench.HEADLINE[2], "projections": bench.HEADLINE[1],
                                                                   "launch": "HIP graph of 20 steps"},
            "roofline": roof, "configs": configs, "next": nexts,
            "ceilings": {"copy_GBs": 5123.123456, "bf16_gemm_TFLOPs": 1390.123456, "int8_gemm_TOPS": 2100.123456},
            "cpu_baseline": cpu}


def test_the_printed_line_is_short_and_whole(tmp_path, monkeypatch, capsys):
    import bench
    out = _record(bench)
    monkeypatch.delenv("BENCH_PHASE_LOG", raising=False)
    monkeypatch.setattr(bench, "PHASE_LOG", [f"{c[0]} {m} {k}" for c in bench.CONFIGS + bench.NEXT for m in ("warm", "cold")
                                             for k in ("call", "quantize", "gemm")])
    details = tmp_path / "d" / "all.json"
    bench.finish(out, 0.0, str(details))
    text = capsys.readouterr().out
    assert text.count("\n") == 1 and len(text) < 4096
    line = json.loads(text)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "config", "roofline"):
        assert line[key] == out[key], key
    ids = [c[0] for c in bench.CONFIGS + bench.NEXT]
    assert list(line["calls_us"]) == ids and line["calls_us"]["C5"] == {"warm": 10.87, "cold": 10.87}
    assert line["calls_us"]["C1"] == {"warm": 10.87} and line["cpu_baseline"]["cores"] == 16
    whole = json.loads(details.read_text())
    assert whole["configs"] == out["configs"] and "profile_phases" in whole


def test_one_workload_prints_its_record(monkeypatch, capsys):
    import bench
    monkeypatch.delenv("BENCH_PHASE_LOG", raising=False)
    configs = _record(bench)["configs"][:1]
    bench.finish({"workload": "C1", "configs": configs}, 0.0)
    assert json.loads(capsys.readouterr().out)["configs"] == configs
