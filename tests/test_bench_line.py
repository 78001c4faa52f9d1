"""The benchmark's line on stdout: the headline's figures, short enough for a
reader of the last 1500 characters, and everything else on stderr."""
import json

import bench


def full_line(long=8):
    """As a run prints it, every figure with all of its digits."""
    x = 12345.678901234567
    kernels = {f"kernel_{i}": {"us": x, "gbs": x, "frac_of_hbm_peak": x} for i in range(long)}
    return {
        "metric": bench.METRIC, "value": x, "unit": "tokens/s", "n_gpus": 8, "steps": 20000, "warmup": 20025,
        "ms_per_step": x, "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
        "dtype": "mxfp8 weights, bf16 activations", "data": "synthetic",
        "config": {"workload": "fwd_t2048_h6144_i2048_e256_k8_bias", "T": 2048, "H": 7168, "I": 2048, "E": 384, "k": 8,
                   "path": "decode_fused", "layers": 100,
                   "l2": "inputs larger than L2: 100 layers' weights (1000.0 GB) cycled step by step, 10000 MB read per "
                         "step at most, fresh tokens per step",
                   "timing": "CUDA graph of the K steps, replayed once untimed and once timed",
                   "parallelism": "replicas x8 (independent token streams)"},
        "roofline": {"kernel": "decode_fused", "kernel_us": kernels}, "call_hbm": {"achieved_gbs": x}, "tensor": {"t": x},
        "cold_call": {"us_median": x}, "gpu_launches": 160000, "stages": ["decode_fused"] * long, "wall_s": x,
        "e2e": {"value": x, "unit": "tokens/s", "h2d_bytes_per_step": 10 ** 9, "d2h_bytes_per_step": 10 ** 9},
        "clocks": {"sm_mhz": 2070.0, "sm_max_mhz": 2070.0, "reasons": ["sw_power_cap"], "samples": 10000,
                   "power_w_max": 1234.56},
        "cpu_baseline": {"value": x}, "supplementary": [kernels] * 20,
    }


def test_the_line_is_one_and_short(capsys):
    line = full_line()
    bench.print_line(line)
    out, err = capsys.readouterr()
    assert out.count("\n") == 1 and len(out) <= bench.LINE_CHARS < 1500
    got = json.loads(out)
    for key in ("metric", "value", "unit", "n_gpus", "steps", "warmup", "ms_per_step", "higher_is_better", "scaling",
                "vs_baseline", "dtype", "data", "e2e", "gpu_launches", "clocks"):
        assert got[key] == line[key], key
    assert got["config"] == {k: v for k, v in line["config"].items() if k != "timing"}
    details = json.loads(err)["details"]
    assert set(details) == {"roofline", "call_hbm", "tensor", "cold_call", "stages", "wall_s", "cpu_baseline",
                            "supplementary", "timing"}
    assert details["supplementary"] == line["supplementary"]


def test_a_line_without_its_optional_parts(capsys):
    line = full_line()
    for key in ("e2e", "supplementary", "cpu_baseline"):
        del line[key]
    bench.print_line(line)
    assert "e2e" not in json.loads(capsys.readouterr()[0])
