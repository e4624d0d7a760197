"""The benchmark's printed line is read from the last 3000 characters of a log: with every
other workload in it, it has to stay below that and keep the keys of the contract."""
import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402

PARITY = {"tokens_compared": 864, "out_f32_max_err_over_rms": 1.3712779237242432e-06,
          "out_bf16_max_err_over_rms": 0.011274951831103452, "bf16_within_bound": True,
          "ids_mismatched": 0, "weights_max_rel_err": 4.9796499494274636e-08,
          "layout_entries_mismatched": 0, "tolerance": "t" * 300, "pass": True}
STAGES = {n: 1.0123456789012345 for n in ("route", "permute", "gather", "w13_gemm_act",
                                          "w2_gemm_weight_combine", "round_bf16")}
CLOCKS = {"sm_mhz": 1965.0, "sm_max_mhz": 1965.0, "reasons": ["sw_power_cap", "sw_thermal"], "samples": 48,
          "source": "nvml every 1 ms, samples inside the timed region"}
ROOF = {"bound": "tensor", "kernel": "grouped_gemm_kernel<0> (w13 + activation)",
        "achieved": 1170.2247698658957, "peak": 1649.5, "unit": "TFLOP/s", "frac": 0.7094421157113645,
        "peak_source": "measured bf16_tflops (burst)", "traffic": 2289897728, "layer_frac": 0.7167374090375672}
CPU = {"value": 400.55276413210817, "unit": "tokens/s", "cores": 16, "kind": "oracle",
       "sample": "864 tokens drawn from the same 4096-token batch in rounds of 16, full layer per token (fp64), 12.1 s"}


def _result():
    entry = {"workload": "w" * 90, "path": "prefill", "ms_per_step": 0.17039840221405028,
             "value": 375590.3762501527, "unit": "tokens/s", "roofline": ROOF, "layer_frac": 0.67,
             "stage_ms": STAGES, "l2": "weights far larger than L2", "parity": PARITY,
             "cpu_baseline": CPU, "clocks": CLOCKS, "gpu_launches": 220}
    return {"metric": bench.METRIC, "value": 1677811.6512972221, "unit": bench.UNIT, "n_gpus": 1, "steps": 20,
            "warmup": 5, "ms_per_step": 2.441275215148926, "higher_is_better": True, "scaling": "weak",
            "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic: seeded N(0,1) tokens, N(0,0.02) bf16 random-init expert weights, fp32 "
                    "router logits with a 1e-3 top-k margin",
            "config": {"workload": "mixtral_prefill: T=4096 H=4096 E=8 k=2 I=14336 SiLU", "path": "prefill",
                       "combine": "fp32 reductions", "timing": "one CUDA-graph replay of the K steps",
                       "global_batch": 4096, "seq_len": 4096, "parallelism": "single",
                       "l2": "inputs larger than L2: the step streams the 2.82 GB of the 8 experts it "
                             "routes to"},
            "roofline": ROOF, "layer_tflops": 1182.3456789, "stage_ms": STAGES, "cpu_baseline": CPU,
            "parity": PARITY,
            "e2e": {"value": 1629435.815598209, "unit": "tokens/s", "h2d_bytes_per_step": 33685504,
                    "d2h_bytes_per_step": 33554432,
                    "timing": "pipelined: input copies, moe_forward and output copies on three streams, "
                              "two buffers each"},
            "gpu_launches": 2400, "clocks": CLOCKS,
            "configs": {name: dict(entry) for name in bench.OTHER_CONFIGS}}


def test_the_line_is_short_and_whole():
    full = _result()
    text = json.dumps(bench.line_of(full))
    assert len(text) < 2900
    line = json.loads(text)
    assert set(line) == set(full)
    assert abs(line["value"] / full["value"] - 1) < 1e-6 and line["e2e"]["h2d_bytes_per_step"] == 33685504
    assert set(line["configs"]) == set(bench.OTHER_CONFIGS)
    assert line["configs"]["decode_t64+fp8"] == {"ms": 0.1704, "frac": 0.709, "parity": True}
    assert "tolerance" in full["parity"]           # the result itself keeps everything


def test_a_result_without_the_other_workloads():
    full = _result()
    del full["configs"]
    full["parity"] = full["cpu_baseline"] = full["e2e"] = None
    assert set(json.loads(json.dumps(bench.line_of(full)))) == set(full)
