"""Benchmark of the SVDQuant W4A4 NVFP4 linear layer on one MI355X.

Workload (default): the DiT FFN w1 projection at 1024^2, M=4096 tokens,
K=3840, N=10240, rank R=128, seeded synthetic inputs (bf16 activations with 1%
outlier channels, NVFP4 weights). One step = one full svdq_linear_w4a4 call
(activation quantisation + down-projection + scaled GEMM + up-projection +
epilogue) with inputs already resident in HBM. Inputs and weights rotate over
several distinct sets (> 512 MB in total) so data comes from HBM, not the
256 MB Infinity Cache.

Prints one JSON line: effective TFLOP/s = (2MNK + 2MR(K+N)) / time per step,
the roofline of the dominant kernel (the GEMM, bound by the f16 matrix cores),
the activation-quantisation kernel's HBM bandwidth, and the CPU oracle timed
on the same workload on the host cores.

Usage: python bench.py [--gpus 1] [--steps 200] [--warmup 50] [--layout packed|canonical]
                       [--workload NAME] [--no-cpu-baseline] [--warm] [--copy-calibration]
"""

import argparse
import hashlib
import json
import math
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "W4A4 SVDQuant linear TFLOP/s and % MFMA peak at M=4096,K=3840,N=10240, 1 GPU"
PEAK_F16_MFMA_TFLOPS = 2500.0   # MI355X dense f16/bf16 matrix peak
PEAK_HBM_GBS = 8000.0           # MI355X HBM3E
CSRC = os.path.join(ROOT, "bit_w4a4_quantized_quantize_amd", "csrc")
GEMM_KERNEL_SOURCES = [os.path.join(CSRC, "gemm_lds.hip"), os.path.join(CSRC, "common.h")]
TRAFFIC_FILE = os.path.join(ROOT, "profiles", "gemm_lds_ffn_w1_1024_traffic.txt")


# name -> (workloads attribute or (dict, key), description). The default is the headline
# workload; the others are the remaining layer shapes of the pages' 1024^2 and 2048px runs.
WORKLOADS = {
    "ffn_w1_1024": ("FFN_W1_1024", "DiT FFN w1 at 1024^2"),
    "ffn_w3_1024": ("FFN_W3_1024", "DiT FFN w3 at 1024^2"),
    "ffn_w2_1024": ("FFN_W2_1024", "DiT FFN w2 at 1024^2 (SwiGLU-like input)"),
    "qkv_1024": ("QKV_1024", "DiT fused QKV projection at 1024^2"),
    "qkv_2048": (("LAYERS_2048", "qkv"), "DiT fused QKV projection at 2048px (16384 image + 512 text tokens)"),
    "out_2048": (("LAYERS_2048", "out"), "DiT attention output projection at 2048px"),
    "ffn_w1_2048": (("LAYERS_2048", "w1"), "DiT FFN w1 at 2048px"),
    "ffn_w2_2048": (("LAYERS_2048", "w2"), "DiT FFN w2 at 2048px"),
    "qkv_1024_tp8": (("SHARDS_TP8_1024", "qkv"), "one GPU's shard of the 1024^2 fused QKV projection at "
                                                 "8-way tensor parallelism (N = 11520 / 8)"),
    "ffn_w1_1024_tp8": (("SHARDS_TP8_1024", "w1"), "one GPU's shard of the 1024^2 FFN w1 at 8-way tensor "
                                                   "parallelism (N = 10240 / 8)"),
    "ffn_w2_1024_tp8": (("SHARDS_TP8_1024", "w2"), "one GPU's shard of the 1024^2 FFN w2 at 8-way tensor "
                                                   "parallelism (K = 10240 / 8, row-parallel)"),
}
DEFAULT_WORKLOAD = "ffn_w1_1024"
# the gated FFN block (w1/w3 as one 2F-channel layer with silu(gate) * up, then w2)
FFN_BLOCKS = {
    "ffn_block_1024": (dict(M=4096, K=3840, N=2 * 10240, R=128, kind="dit", seed=1003), "FFN_W2_1024",
                       "DiT FFN block at 1024^2"),
    # one GPU's share under 8-way tensor parallelism: w1/w3 by columns (F = 1280), w2 by rows
    "ffn_block_1024_tp8": (dict(M=4096, K=3840, N=2 * 1280, R=128, kind="dit", seed=1053),
                           ("SHARDS_TP8_1024", "w2"), "one GPU's share of the DiT FFN block at 1024^2 under "
                           "8-way tensor parallelism (F = 10240 / 8)"),
}


# the attention half of a DiT block between two norms: tokens, width, heads, text tokens
ATTN_BLOCKS = {
    "attn_block_1024": (dict(M=4096, K=3840, H=30, text=0), "DiT attention half-block at 1024^2"),
    "attn_block_2048": (dict(M=16384 + 512, K=3840, H=30, text=512),
                        "DiT attention half-block at 2048px (16384 image + 512 text tokens)"),
}


# the mixed-precision linear sweep of a whole DiT forward (bf16 and W4A4 layers)
SWEEPS = {
    "dit_sweep_1024": "DiT mixed-precision linear sweep at 1024^2: 30 blocks x {qkv, out, w1, w3, w2}, "
                      "M=4096; qkv/out of every block and all linears of blocks 0-4 and 25-29 in bf16, "
                      "the other 60 FFN linears SVDQuant W4A4 NVFP4 R=128; one step = one forward (150 "
                      "linears) with fresh activations, cycling over 8 forwards",
}


# load-time SVDQuant preparation of one weight (the FFN w1 shape at 1024^2)
PREPS = {
    "prep_ffn_w1_1024": dict(N=10240, K=3840, R=128, iters=2, seed=1003,
                             desc="SVDQuant weight preparation of a DiT FFN w1 weight (N=10240, K=3840, R=128, "
                                  "2 power rounds): randomized rank-R split, residual, two-level scales, NVFP4 codes"),
}
PEAK_FP64_TFLOPS = 78.6    # MI355X fp64 vector peak
PEAK_FP4_MFMA_TFLOPS = 10100.0   # MI355X dense FP4 matrix peak
# the MXFP4 datatype variant of a layer shape (out of the pages' tolerance: a speed point)
MX_VARIANTS = {"ffn_w1_1024_mxfp4": "ffn_w1_1024", "qkv_1024_mxfp4": "qkv_1024", "ffn_w2_1024_mxfp4": "ffn_w2_1024"}


# the static (calibrated) activation-scale variant of a layer shape, beside the dynamic layer
STATIC_VARIANTS = {"ffn_w1_1024_static": "ffn_w1_1024", "ffn_w2_1024_static": "ffn_w2_1024",
                   "qkv_1024_static": "qkv_1024"}


def run_static(args):
    """Static activation scales: g calibrated by the library on a separate seeded batch of the
    same distribution; the layer timed like the headline; accuracy of the static and the dynamic
    layer against the unquantised float64 product on sampled rows."""
    import numpy as np
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops
    from oracle import formats as Fm

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    cfg, desc = workload_cfg(STATIC_VARIANTS[args.workload])
    M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]
    n_sets = 1 if args.warm else args.sets
    print(f"[bench] static activation scales: building {n_sets} sets for M={M} K={K} N={N} R={R}",
          file=sys.stderr, flush=True)
    d, sets = make_sets(cfg, n_sets, "packed", dev)
    cal = workloads.make_linear(**dict(cfg, seed=cfg["seed"] + 1000))

    def bf(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(dev)

    g = ops.calibrate_act_gscale(bf(cal["x"]), sets[0]["layer"].smooth)
    torch.cuda.synchronize()
    g_val = float(g.float().item())
    flops = 2 * M * N * K + 2 * M * R * (K + N)

    def step(i):
        st = sets[i]
        ops.linear_w4a4_static(st["x"], st["layer"], g, y=st["y"], workspace=st["ws"])

    ms, cond = timed(step, n_sets, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    tflops = flops / (ms * 1e-3) / 1e12
    dyn_ms = time_loop(lambda i: ops.linear_w4a4(sets[i]["x"], sets[i]["layer"], y=sets[i]["y"],
                                                 workspace=sets[i]["ws"]), n_sets, args.kernel_iters, 1, stream)
    st = sets[0]
    y_s = ops.linear_w4a4_static(st["x"], st["layer"], g)
    y_d = ops.linear_w4a4(st["x"], st["layer"])
    qa, sa, _ = ops.quantize_act_static(st["x"], st["layer"].smooth, g)
    torch.cuda.synchronize()
    sat = float((sa == 0x7E).float().mean().item())
    dist = float(torch.linalg.vector_norm(y_s.float() - y_d.float()) / torch.linalg.vector_norm(y_d.float()))
    # accuracy against the unquantised layer (x * smooth) W^T + (x proj_down) proj_up^T + bias on sampled rows
    rows = np.sort(np.random.default_rng(7).choice(M, size=min(256, M), replace=False))
    x64 = Fm.bf16_to_f64(d["x"][rows])
    ref = (x64 * Fm.bf16_to_f64(d["smooth"])[None, :]) @ np.asarray(d["W"], np.float64).T
    ref = ref + (x64 @ Fm.bf16_to_f64(d["proj_down"])) @ Fm.bf16_to_f64(d["proj_up"]).T + Fm.bf16_to_f64(d["bias"])
    rsel = torch.from_numpy(rows).to(dev)

    def err(y):
        yy = y.index_select(0, rsel).float().cpu().double().numpy()
        return float(np.linalg.norm(yy - ref) / np.linalg.norm(ref))

    e_s, e_d = err(y_s), err(y_d)
    print(f"[bench] static layer {ms * 1e3:.1f} us ({tflops:.1f} TFLOP/s), dynamic {dyn_ms * 1e3:.1f} us; g = {g_val:.6g}; "
          f"saturated block scales {sat:.2e}; static vs dynamic {dist:.4f}; error vs unquantised: static {e_s:.4f}, "
          f"dynamic {e_d:.4f}", file=sys.stderr, flush=True)
    result = {
        "metric": f"SVDQuant W4A4 linear with static (calibrated) activation scales, TFLOP/s at M={M},K={K},N={N}, 1 GPU",
        "value": round(tflops, 2), "unit": "TFLOP/s", "n_gpus": 1, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": round(ms, 5), "higher_is_better": True, "scaling": "weak", "vs_baseline": None,
        "dtype": "f16", "data": "synthetic",
        "config": {"workload": f"{desc}: static global activation scale calibrated on another seeded batch "
                               f"(seed {cfg['seed'] + 1000}), per-16 e4m3 block scales relative to it; "
                               f"M={M} K={K} N={N} R={R}",
                   "cache": "warm" if args.warm else f"cold (rotating {n_sets} sets)",
                   **({"gemm_tile_forced": args.gemm_tile} if args.gemm_tile else {})},
        "act_gscale": g_val, "saturated_block_scale_fraction": sat,
        "dynamic_layer_us": round(dyn_ms * 1e3, 2),
        "normwise_static_vs_dynamic": round(dist, 5),
        "error_vs_unquantised": {"static": round(e_s, 5), "dynamic": round(e_d, 5), "rows": len(rows)},
        "conditioning": cond,
    }
    print(json.dumps(result), flush=True)


# roofline calibration of this device (no layer): sustained f16 MFMA and device copy
CALIBS = {"calib": "sustained v_mfma_f32_32x32x16_f16 (8 waves per CU, the GEMM's occupancy and accumulator "
                   "footprint) on exact NVFP4 values, random f16 bits and zeros, and the block-scaled "
                   "v_mfma_scale_f32_32x32x64_f8f6f4 on random fp4 and fp8 operands, with the shader clock read "
                   "by the kernel; streaming device copy of 1 GiB (HBM) and 64 MiB (cache resident); LDS "
                   "bandwidth of 16-byte reads, writes and a 3:1 mix"}


# the oracle's own timing on the host cores (no GPU): the configurations of the pages'
# workloads, quantisation and the rest of the layer timed apart
ORACLE_TIMES = {"oracle_times": "the CPU oracle (NumPy float64 / int64) per layer call: median of 3 at the "
                                "tiny config, the 1024^2 QKV and FFN w1 layers; one run per 2048px layer; the "
                                "mixed-precision forward extrapolated from per-layer rates"}


def blas_info():
    try:
        from threadpoolctl import threadpool_info
        info = threadpool_info()
        return [{k: i.get(k) for k in ("internal_api", "num_threads", "version")} for i in info]
    except Exception:
        return []


def run_oracle_times(args):
    import numpy as np

    import workloads
    from oracle import svdq as S

    cfgs = [("tiny", dict(workloads.TINY), 3), ("qkv_1024", dict(workloads.QKV_1024), 3),
            ("ffn_w1_1024", dict(workloads.FFN_W1_1024), 3)]
    cfgs += [(f"{k}_2048", dict(v), 1) for k, v in workloads.LAYERS_2048.items()]
    rows = {}
    for name, cfg, reps in cfgs:
        d = workloads.make_linear(**cfg)
        qw, ws = S.quantize_weight(d["W"], d["wcscales"], d["wtscale"])   # load time, not timed
        M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]
        tq, tr = [], []
        for _ in range(reps):
            t0 = time.perf_counter()
            qact, asc = S.quantize_act(d["x"], d["smooth"])
            t1 = time.perf_counter()
            main = S.main_term(qact, asc, qw, ws)
            lr = S.lowrank(d["x"], d["proj_down"], d["proj_up"])
            S.epilogue(main, d["wcscales"], d["wtscale"], lr, d["bias"])
            t2 = time.perf_counter()
            tq.append(t1 - t0)
            tr.append(t2 - t1)
            del qact, asc, main, lr
        q, r = float(np.median(tq)), float(np.median(tr))
        flops = 2 * M * N * K + 2 * M * R * (K + N)
        qbytes = M * K * 2 + K * 2 + M * K // 2 + (K // 16) * M
        rows[name] = {"M": M, "K": K, "N": N, "R": R, "runs": reps, "quant_s": round(q, 4), "rest_s": round(r, 4),
                      "layer_s": round(q + r, 4), "TFLOPs": round(flops / (q + r) / 1e12, 4),
                      "quant_GBps": round(qbytes / q / 1e9, 3)}
        print(f"[oracle] {name}: {rows[name]}", file=sys.stderr, flush=True)
        del d, qw, ws
    # one bf16 layer (the out projection at 1024^2), then the mixed-precision forward
    # (90 bf16 + 60 W4A4 linears at M=4096) extrapolated from the measured per-flop rates
    db = workloads.make_bf16_linear(4096, 3840, 3840, kind="dit", seed=5001)
    t0 = time.perf_counter()
    S.linear_bf16(db["x"], db["W"], db["bias"])
    t_bf = time.perf_counter() - t0
    rate_bf = 2 * 4096 * 3840 * 3840 / t_bf
    rows["out_1024_bf16"] = {"M": 4096, "K": 3840, "N": 3840, "runs": 1, "layer_s": round(t_bf, 4),
                             "TFLOPs": round(rate_bf / 1e12, 4)}
    print(f"[oracle] out_1024_bf16: {rows['out_1024_bf16']}", file=sys.stderr, flush=True)
    t_fwd = 0.0
    for L in workloads.sweep_layers():
        if L["precision"] == "bf16":
            t_fwd += 2 * 4096 * L["K"] * L["N"] / rate_bf
        else:
            rate = rows["ffn_w1_1024" if L["K"] == 3840 else "w2_2048"]["TFLOPs"] * 1e12
            t_fwd += (2 * 4096 * L["K"] * L["N"] + 2 * 4096 * 128 * (L["K"] + L["N"])) / rate
    cores = len(os.sched_getaffinity(0))
    result = {
        "metric": "CPU oracle seconds per SVDQuant W4A4 linear call at M=4096,K=3840,N=10240 (host cores)",
        "value": rows["ffn_w1_1024"]["layer_s"],
        "unit": "s",
        "n_gpus": 0,
        "steps": 3,
        "warmup": 0,
        "ms_per_step": rows["ffn_w1_1024"]["layer_s"] * 1e3,
        "higher_is_better": False,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f64",
        "data": "synthetic",
        "config": {"workload": ORACLE_TIMES["oracle_times"], "cores": cores,
                   "OMP_NUM_THREADS": os.environ.get("OMP_NUM_THREADS"), "blas": blas_info()},
        "layers": rows,
        "mixed_precision_forward_s_extrapolated": round(t_fwd, 1),
    }
    print(json.dumps(result), flush=True)


def run_calib(args):
    import torch
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    res = calibration(dev, stream)
    for k, v in res.items():
        print(f"[bench] {k}: {v}", file=sys.stderr, flush=True)
    m = res["mfma_f16_32x32x16"]
    result = {
        "metric": "MI355X roofline calibration: sustained f16 MFMA TFLOP/s on exact NVFP4 operand values, 1 GPU",
        "value": m["nvfp4_values"]["TFLOPs"],
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": 1,
        "warmup": 0,
        "ms_per_step": m["nvfp4_values"]["ms_per_launch"],
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f16",
        "data": "synthetic",
        "config": {"workload": CALIBS["calib"]},
        "published_peaks": {"f16_mfma_TFLOPs": PEAK_F16_MFMA_TFLOPS, "hbm_GBps": PEAK_HBM_GBS},
        "calibration": res,
    }
    print(json.dumps(result), flush=True)


def workload_cfg(name):
    import workloads
    ref, desc = WORKLOADS[name]
    cfg = getattr(workloads, ref) if isinstance(ref, str) else getattr(workloads, ref[0])[ref[1]]
    return dict(cfg), desc


def parse():
    p = argparse.ArgumentParser()
    p.add_argument("--workload",
                   choices=sorted(WORKLOADS) + sorted(FFN_BLOCKS) + sorted(SWEEPS) + sorted(PREPS) + sorted(MX_VARIANTS)
                   + sorted(CALIBS) + sorted(ORACLE_TIMES) + sorted(STATIC_VARIANTS) + sorted(ATTN_BLOCKS),
                   default=DEFAULT_WORKLOAD,
                   help="layer shape (the default is the headline workload; the rest are for comparison)")
    p.add_argument("--gpus", type=int, default=1)
    p.add_argument("--steps", type=int, default=200)
    p.add_argument("--warmup", type=int, default=50,
                   help="untimed steps first (the chip takes ~15 ms of matrix work to reach its sustained clock)")
    p.add_argument("--layout", choices=["packed", "canonical"], default="packed")
    p.add_argument("--sets", type=int, default=6, help="distinct input/weight sets rotated (cold cache)")
    p.add_argument("--warm", action="store_true", help="reuse one set (warm cache)")
    p.add_argument("--no-cpu-baseline", action="store_true")
    p.add_argument("--kernel-iters", type=int, default=100)
    p.add_argument("--no-graph", action="store_true", help="sweep: time eager launches only")
    p.add_argument("--copy-calibration", action="store_true",
                   help="finish with a plain 512 MiB device copy (to calibrate HBM byte counters)")
    p.add_argument("--gemm-tile", type=int, default=0, choices=[0, 1, 2, 3, 4],
                   help="force the W4A4 GEMM's tile shape (0 automatic, 1 256x320, 2 256x256, 3 128x320, "
                        "4 128x160), for comparisons")
    p.add_argument("--condition-ms", type=float, default=30.0,
                   help="minimum untimed device work before timing; conditioning also waits until "
                        "consecutive ~2 ms windows agree within 2%%")
    return p.parse_args()


def source_hash(paths):
    h = hashlib.sha256()
    for path in paths:
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def read_traffic():
    """HBM bytes per GEMM launch from the committed rocprofv3 --pmc summary, if it was
    taken on the current kernel source; otherwise None."""
    if not os.path.exists(TRAFFIC_FILE):
        return None
    vals = {}
    with open(TRAFFIC_FILE) as f:
        for line in f:
            if ":" in line and not line.startswith("#"):
                k, v = line.split(":", 1)
                vals[k.strip()] = v.strip()
    if vals.get("kernel_source_sha256") != source_hash(GEMM_KERNEL_SOURCES):
        return None
    try:
        return float(vals["hbm_bytes_per_launch"])
    except (KeyError, ValueError):
        return None


def make_sets(cfg, n_sets, layout, dev):
    """Device tensors for n_sets copies of the layer (distinct addresses, same values)."""
    import numpy as np
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    d = workloads.make_linear(**cfg)
    M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]

    def bf(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(dev)

    wc = bf(d["wcscales"])
    wt = bf(d["wtscale"])
    # NVFP4 weight from the library's own quantiser: W' = W / (wtscale * wcscales) in fp32,
    # rounded to bf16, quantised per 16-block with smooth = 1.
    W = torch.from_numpy(d["W"]).to(dev)
    Wp = (W / (wt.float() * wc.float())[:, None]).to(torch.bfloat16).contiguous()
    ones = torch.ones(K, dtype=torch.bfloat16, device=dev)
    qweight, wscales, _ = ops.quantize_act(Wp, ones)
    del W, Wp
    base = ops.SVDQLinearWeights(N=N, K=K, weight=qweight, wscales=wscales, wcscales=wc, wtscale=wt,
                                 smooth=bf(d["smooth"]), proj_down=bf(d["proj_down"]),
                                 proj_up=bf(d["proj_up"]), bias=bf(d["bias"]))
    if layout == "packed":
        base = base.packed()
    x0 = bf(d["x"])
    sets = []
    ws_bytes = ops.linear_workspace_bytes(M, N, K, R)
    for i in range(n_sets):
        layer = ops.SVDQLinearWeights(
            N=N, K=K, weight=base.weight.clone(), wscales=None if base.wscales is None else base.wscales.clone(),
            wcscales=base.wcscales.clone(), wtscale=base.wtscale.clone(), smooth=base.smooth.clone(),
            proj_down=base.proj_down.clone(), proj_up=base.proj_up.clone(), bias=base.bias.clone(),
            layout=base.layout)
        sets.append(dict(
            x=x0.clone(), layer=layer,
            y=torch.empty((M, N), dtype=torch.bfloat16, device=dev),
            ws=torch.empty(ws_bytes, dtype=torch.uint8, device=dev),
            qact=torch.empty((M, K // 2), dtype=torch.uint8, device=dev),
            ascales=torch.empty((K // 16, M), dtype=torch.uint8, device=dev),
            qpk=torch.empty(ops._lib.lib().svdq_packed_act_bytes(M, K), dtype=torch.uint8, device=dev),
            lora=torch.empty((M, R), dtype=torch.bfloat16, device=dev)))
    return d, sets


def condition(fn, n_sets, stream, min_ms=30.0, window_ms=2.0, tol=0.02, max_ms=3000.0):
    """Run fn(set_index) untimed until at least min_ms of device work has run and two
    consecutive windows of about window_ms agree within tol: under sustained matrix work the
    chip settles its clock over some milliseconds, so a fixed number of warm-up calls
    conditions it differently for different call lengths. The device never idles between
    windows (the host waits for a window only after queueing the next one); the last
    window is still running when this returns. Returns (conditioning_ms, calls, window
    times in ms per call)."""
    import torch
    ev = lambda: torch.cuda.Event(enable_timing=True)   # noqa: E731
    a, b = ev(), ev()
    a.record(stream)
    fn(0)
    b.record(stream)
    b.synchronize()
    est = max(a.elapsed_time(b), 1e-3)
    per = max(1, int(round(window_ms / est)))
    calls = 1
    total = est

    def enqueue():
        nonlocal calls
        s, e = ev(), ev()
        s.record(stream)
        for _ in range(per):
            fn(calls % n_sets)
            calls += 1
        e.record(stream)
        return s, e

    times = []
    pending = enqueue()
    while True:
        nxt = enqueue()
        pending[1].synchronize()
        t = pending[0].elapsed_time(pending[1]) / per
        times.append(t)
        total += t * per
        pending = nxt
        settled = len(times) >= 2 and abs(times[-1] - times[-2]) <= tol * times[-2]
        if (total >= min_ms and settled) or total >= max_ms:
            break
    total += times[-1] * per    # the window still in flight
    return total, calls, times


def timed(fn, n_sets, iters, stream, warmup=0, min_ms=30.0):
    """Average ms per call of fn(set_index) over `iters` calls on `stream`: conditioning by
    time, `warmup` more untimed calls, a host synchronisation, about 1 ms of untimed calls
    queued ahead of the start event (so the timed calls start on a busy device), then HIP
    events around exactly `iters` calls. Python's cyclic garbage collector is run once
    beforehand and kept off until the end (as timeit does): a full collection in the middle
    of the timed calls stops the host for tens of milliseconds, and the device then idles.
    Returns (ms per call, info)."""
    import gc
    gc_on = gc.isenabled()
    gc.collect()
    gc.disable()
    try:
        return _timed(fn, n_sets, iters, stream, warmup, min_ms)
    finally:
        if gc_on:
            gc.enable()


def _timed(fn, n_sets, iters, stream, warmup, min_ms):
    import torch
    cond_ms, cond_calls, windows = condition(fn, n_sets, stream, min_ms=min_ms)
    for i in range(warmup):
        fn(i % n_sets)
    torch.cuda.synchronize()
    per_call = windows[-1]
    prime = max(1, int(round(1.0 / max(per_call, 1e-3))))
    for i in range(prime):
        fn(i % n_sets)
    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    start.record(stream)
    for i in range(iters):
        fn(i % n_sets)
    end.record(stream)
    torch.cuda.synchronize()
    info = {"conditioning_ms": round(cond_ms + prime * per_call, 2), "conditioning_calls": cond_calls + prime,
            "conditioning_windows_us": [round(t * 1e3, 1) for t in windows[-4:]]}
    return start.elapsed_time(end) / iters, info


def step_percentiles(fn, n_sets, iters, stream):
    """p10 / p50 / p90 of the per-call device time of fn(set_index) over `iters` back-to-back
    calls, from one HIP event recorded between consecutive calls (the calls are all queued
    before the host waits, so the device runs them back to back). A separate pass after the
    timed region, conditioned by time like it and started while the conditioning calls still
    run: the events do not touch the headline figure. Microseconds."""
    import gc

    import numpy as np
    import torch
    gc_on = gc.isenabled()
    gc.collect()
    gc.disable()
    try:
        evs = [torch.cuda.Event(enable_timing=True) for _ in range(iters + 1)]
        condition(fn, n_sets, stream, min_ms=10.0)
        evs[0].record(stream)
        for i in range(iters):
            fn(i % n_sets)
            evs[i + 1].record(stream)
        torch.cuda.synchronize()
    finally:
        if gc_on:
            gc.enable()
    t = np.array([evs[i].elapsed_time(evs[i + 1]) * 1e3 for i in range(iters)])
    return {"p10": round(float(np.percentile(t, 10)), 2), "p50": round(float(np.percentile(t, 50)), 2),
            "p90": round(float(np.percentile(t, 90)), 2), "n": iters,
            "note": "one event between consecutive calls; the events add a few us per call, so these sit "
                    "slightly above the mean of the event-pair timing"}


def device_info(dev):
    """Compute units and clock as the runtime reports them (the published peaks assume 256 CUs
    at 2.4 GHz)."""
    import torch
    pr = torch.cuda.get_device_properties(dev)
    info = {"name": pr.name, "compute_units": pr.multi_processor_count,
            "arch": getattr(pr, "gcnArchName", None)}
    clk = getattr(pr, "clock_rate", None)
    if clk:
        info["max_clock_MHz"] = round(clk / 1000.0, 1)
    return info


def time_loop(fn, n_sets, iters, warmup, stream):
    """Average ms per call of fn(set_index) on `stream` (conditioned by time; see timed)."""
    return timed(fn, n_sets, iters, stream, warmup=warmup, min_ms=10.0)[0]


# ---- roofline calibration (measurement helpers in the library) ----

def calib_tables(dev):
    """Operand tables for the sustained-MFMA kernel: f16 values with random bits (sign,
    exponents 2^-4..2^3, all 10 mantissa bits), exact NVFP4 values (E2M1 code times an
    e4m3 block scale, as the GEMM multiplies them), and zeros."""
    import torch
    from bit_w4a4_quantized_quantize_amd import _lib
    n = _lib.lib().svdq_calib_table_bytes() // 2
    g = torch.Generator(device="cpu").manual_seed(2024)
    sign = torch.randint(0, 2, (n,), generator=g) * 2 - 1
    expo = torch.randint(-4, 4, (n,), generator=g).double()
    mant = 1.0 + torch.randint(0, 1024, (n,), generator=g).double() / 1024.0
    rnd = (sign * mant * torch.pow(2.0, expo)).to(torch.float16)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    code = torch.randint(0, 16, (n,), generator=g)
    e2m1 = torch.where(code >= 8, -grid[code % 8], grid[code % 8])
    # e4m3 scales of a typical block: exponent 2^-3..2^2, any 3-bit mantissa
    sc = (1.0 + torch.randint(0, 8, (n // 16,), generator=g).double() / 8.0) * \
        torch.pow(2.0, torch.randint(-3, 3, (n // 16,), generator=g).double())
    nv = (e2m1 * sc.repeat_interleave(16)).to(torch.float16)
    # bytes for the block-scaled instruction: any byte is a pair of valid E2M1 codes; for e4m3
    # the two NaN patterns (S.1111.111) are moved to the largest finite magnitude
    byts = torch.randint(0, 256, (2 * n,), generator=g, dtype=torch.int64)
    fp8 = torch.where((byts & 0x7F) == 0x7F, byts - 1, byts)
    return {"random_f16": rnd.to(dev), "nvfp4_values": nv.to(dev), "zeros": torch.zeros(n, dtype=torch.float16,
                                                                                         device=dev),
            "random_fp4_codes": byts.to(torch.uint8).to(dev), "random_fp8_e4m3": fp8.to(torch.uint8).to(dev)}


def calib_mfma(table, dev, stream, target_ms=20.0, workgroups=256, fmt=None):
    """Sustained MFMA rate on `table`, conditioned by time: v_mfma_f32_32x32x16_f16 (fmt None)
    or the block-scaled v_mfma_scale_f32_32x32x64_f8f6f4 with both operands in format fmt
    (4 = fp4, 0 = fp8); returns TFLOP/s and the median shader clock (GHz) from the kernel's
    own counters."""
    import torch
    from bit_w4a4_quantized_quantize_amd import _lib
    L = _lib.lib()
    out = torch.empty(workgroups * 512, dtype=torch.float32, device=dev)
    clocks = torch.zeros(workgroups * 4, dtype=torch.int64, device=dev)
    nbytes = table.numel() * table.element_size()
    if fmt is None:
        per_iter = L.svdq_calib_flop_per_iteration(workgroups)
    else:
        per_iter = L.svdq_calib_scaled_flop_per_iteration(workgroups)

    def launch(iters):
        if fmt is None:
            _lib.check("svdq_calib_mfma", L.svdq_calib_mfma(table.data_ptr(), nbytes, iters, workgroups,
                                                            out.data_ptr(), out.numel() * 4, clocks.data_ptr(),
                                                            clocks.numel() * 8, stream.cuda_stream))
        else:
            _lib.check("svdq_calib_mfma_scaled",
                       L.svdq_calib_mfma_scaled(table.data_ptr(), nbytes, iters, workgroups, fmt, out.data_ptr(),
                                                out.numel() * 4, clocks.data_ptr(), clocks.numel() * 8,
                                                stream.cuda_stream))

    rate = 1.6e15 if fmt is None else 6.0e15
    iters = max(1, int(2.0 * rate * 1e-3 / per_iter))     # about 2 ms per launch
    ms, info = timed(lambda i: launch(iters), 1, max(1, int(target_ms / 2.0)), stream, min_ms=30.0)
    tflops = iters * per_iter / (ms * 1e-3) / 1e12
    launch(iters)
    torch.cuda.synchronize()
    khz = ctypes_int()
    _lib.check("svdq_calib_wall_clock_khz", L.svdq_calib_wall_clock_khz(khz))
    c = clocks.view(workgroups, 4).cpu().double()
    ghz = ((c[:, 1] - c[:, 0]) / (c[:, 3] - c[:, 2]) * khz.value * 1e3 / 1e9).median().item()
    return {"TFLOPs": round(tflops, 1), "shader_clock_GHz": round(ghz, 3), "ms_per_launch": round(ms, 4),
            "flop_per_launch": iters * per_iter, "workgroups": workgroups, "wall_clock_kHz": khz.value}


def ctypes_int():
    import ctypes
    return ctypes.c_int(0)


def calib_copy(dev, stream, nbytes, reps=10):
    """Device-copy rate (bytes read + written per second) of a streaming copy kernel."""
    import torch
    from bit_w4a4_quantized_quantize_amd import _lib
    L = _lib.lib()
    src = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    src.random_(0, 256)
    dst = torch.empty_like(src)

    def f(i):
        _lib.check("svdq_calib_copy", L.svdq_calib_copy(src.data_ptr(), dst.data_ptr(), nbytes, stream.cuda_stream))

    ms, _ = timed(f, 1, reps, stream, min_ms=10.0)
    del src, dst
    return round(2 * nbytes / (ms * 1e-3) / 1e9, 1), round(ms * 1e3, 2)


def calib_lds(dev, stream, mode, workgroups=256):
    """Chip-wide LDS bandwidth (TB/s of bytes moved) of 16-byte accesses: mode 0 reads, 1
    writes, 2 three reads to one write."""
    import torch
    from bit_w4a4_quantized_quantize_amd import _lib
    L = _lib.lib()
    out = torch.empty(workgroups * 512, dtype=torch.float32, device=dev)
    per_iter = L.svdq_calib_lds_bytes_per_iteration(workgroups)
    iters = 4096

    def launch(i):
        _lib.check("svdq_calib_lds", L.svdq_calib_lds(iters, workgroups, mode, out.data_ptr(), out.numel() * 4,
                                                      stream.cuda_stream))

    ms, _ = timed(launch, 1, 10, stream, min_ms=10.0)
    return {"TBps": round(iters * per_iter / (ms * 1e-3) / 1e12, 1), "ms_per_launch": round(ms, 4),
            "bytes_per_launch": iters * per_iter}


def calibration(dev, stream, quick=False):
    """Sustained f16 MFMA rates and device-copy rates on this device."""
    tables = calib_tables(dev)
    res = {"mfma_f16_32x32x16": {}}
    for name in (("nvfp4_values", "random_f16") if quick else ("nvfp4_values", "random_f16", "zeros")):
        res["mfma_f16_32x32x16"][name] = calib_mfma(tables[name], dev, stream)
    if not quick:
        res["mfma_scaled_32x32x64"] = {
            "fp4_random_codes": calib_mfma(tables["random_fp4_codes"], dev, stream, fmt=4),
            "fp8_e4m3_random": calib_mfma(tables["random_fp8_e4m3"], dev, stream, fmt=0)}
    gbs, us = calib_copy(dev, stream, 1 << 30)
    res["copy_1GiB"] = {"GBps": gbs, "us": us}
    if not quick:
        gbs, us = calib_copy(dev, stream, 64 << 20, reps=50)
        res["copy_64MiB_cache_resident"] = {"GBps": gbs, "us": us}
        res["lds_16B_accesses"] = {"reads": calib_lds(dev, stream, 0), "writes": calib_lds(dev, stream, 1),
                                   "three_reads_one_write": calib_lds(dev, stream, 2)}
    return res


def cpu_baseline(d, cfg, repeats=5):
    """The oracle (untuned NumPy float64) on the same workload, whole layer per call: five
    calls (about 10 s of host work at the headline shape), median."""
    import numpy as np
    from oracle import svdq as S

    qw, ws = S.quantize_weight(d["W"], d["wcscales"], d["wtscale"])   # load-time, not timed
    times = []
    for _ in range(repeats):
        t0 = time.perf_counter()
        S.linear_w4a4(d["x"], d["smooth"], qw, ws, d["wcscales"], d["wtscale"],
                      d["proj_down"], d["proj_up"], d["bias"])
        times.append(time.perf_counter() - t0)
    t = float(np.median(times))
    M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]
    flops = 2 * M * N * K + 2 * M * R * (K + N)
    try:
        from threadpoolctl import threadpool_info
        threads = max([i.get("num_threads", 1) for i in threadpool_info()] or [1])
    except Exception:
        threads = len(os.sched_getaffinity(0))
    return {"value": flops / t / 1e12, "unit": "TFLOP/s", "cores": int(threads), "kind": "oracle",
            "sample": f"the whole layer call (M={M} K={K} N={N} R={R}), median of {repeats}; "
                      f"{t:.2f} s per call; weight quantisation excluded (load time)",
            "seconds_per_call": t}


def cpu_baseline_ffn(d13, d2, F_out):
    """The oracle on one FFN block call (gated w1/w3 then w2), weights quantised beforehand."""
    import numpy as np
    from oracle import formats as Fm
    from oracle import svdq as S

    qw13, ws13 = S.quantize_weight(d13["W"], d13["wcscales"], d13["wtscale"])
    qw2, ws2 = S.quantize_weight(d2["W"], d2["wcscales"], d2["wtscale"])
    t0 = time.perf_counter()
    _, h = S.linear_w4a4_swiglu(d13["x"], d13["smooth"], qw13, ws13, d13["wcscales"], d13["wtscale"],
                                d13["proj_down"], d13["proj_up"], d13["bias"])
    S.linear_w4a4(h, d2["smooth"], qw2, ws2, d2["wcscales"], d2["wtscale"], d2["proj_down"], d2["proj_up"],
                  d2["bias"])
    t = time.perf_counter() - t0
    try:
        from threadpoolctl import threadpool_info
        threads = max([i.get("num_threads", 1) for i in threadpool_info()] or [1])
    except Exception:
        threads = len(os.sched_getaffinity(0))
    del np, Fm
    return t, int(threads)


def run_ffn_block(args):
    """The gated FFN block: h = silu(x W1^T) * (x W3^T) by one gated call, then y = w2(h)."""
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    cfg13, w2_name, desc = FFN_BLOCKS[args.workload]
    cfg2 = dict(getattr(workloads, w2_name) if isinstance(w2_name, str)
                else getattr(workloads, w2_name[0])[w2_name[1]])
    M, K, R = cfg13["M"], cfg13["K"], cfg13["R"]
    F_out = cfg13["N"] // 2
    N2 = cfg2["N"]
    assert cfg2["K"] == F_out and cfg2["M"] == M
    n_sets = 1 if args.warm else args.sets
    print(f"[bench] building {n_sets} input sets: gated M={M} K={K} F={F_out}, w2 K={F_out} N={N2}, R={R}",
          file=sys.stderr, flush=True)
    d13, sets13 = make_sets(cfg13, n_sets, "packed", dev)
    d2, sets2 = make_sets(cfg2, n_sets, "packed", dev)
    hs = [torch.empty((M, F_out), dtype=torch.bfloat16, device=dev) for _ in range(n_sets)]
    torch.cuda.synchronize()

    flops13 = 2 * M * (2 * F_out) * K + 2 * M * R * (K + 2 * F_out)
    flops2 = 2 * M * N2 * F_out + 2 * M * R * (F_out + N2)
    flops_block = flops13 + flops2
    flops_gated_gemm = 2 * M * (2 * F_out) * K + 2 * M * (2 * F_out) * R

    def step(i):
        a, b = sets13[i], sets2[i]
        ops.linear_w4a4_gated(a["x"], a["layer"], h=hs[i], workspace=a["ws"])
        ops.linear_w4a4(hs[i], b["layer"], y=b["y"], workspace=b["ws"])

    t0 = time.perf_counter()
    ms_per_step, cond = timed(step, n_sets, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    wall = time.perf_counter() - t0
    tflops = flops_block / (ms_per_step * 1e-3) / 1e12
    print(f"[bench] FFN block: {ms_per_step * 1e3:.1f} us/step, {tflops:.1f} TFLOP/s "
          f"(conditioned {cond['conditioning_ms']:.1f} ms; wall {wall:.2f} s)", file=sys.stderr, flush=True)

    # per-kernel: the gated GEMM alone (packed activations, as inside the block)
    for i in range(n_sets):
        a = sets13[i]
        ops.quantize_act(a["x"], a["layer"].smooth, a["layer"].proj_down, qact=a["qpk"], lora_act=a["lora"],
                         packed=True)
    torch.cuda.synchronize()

    def gated_gemm(i):
        a = sets13[i]
        ops.gemm_w4a4_gated(a["qpk"], a["lora"], a["layer"], M, h=hs[i])

    def w2_layer(i):
        b = sets2[i]
        ops.linear_w4a4(hs[i], b["layer"], y=b["y"], workspace=b["ws"])

    def unfused(i):
        # the same block without the gated epilogue: the 2F-channel layer's bf16
        # output, the gate as separate elementwise work, then w2
        a, b = sets13[i], sets2[i]
        y = ops.linear_w4a4(a["x"], a["layer"])
        h = torch.nn.functional.silu(y[:, :F_out].float()).mul_(y[:, F_out:].float()).to(torch.bfloat16)
        ops.linear_w4a4(h, b["layer"], y=b["y"], workspace=b["ws"])

    # the block with w2's input quantised in the gated epilogue: quantise x (+ down), the gated
    # GEMM that also writes w2's packed codes, w2's down-projection alone, w2's GEMM
    q13 = [torch.empty(ops._lib.lib().svdq_packed_act_bytes(M, K), dtype=torch.uint8, device=dev)
           for _ in range(n_sets)]
    l13 = [torch.empty((M, R), dtype=torch.bfloat16, device=dev) for _ in range(n_sets)]
    q2 = [torch.empty(ops._lib.lib().svdq_packed_act_bytes(M, F_out), dtype=torch.uint8, device=dev)
          for _ in range(n_sets)]
    l2 = [torch.empty((M, R), dtype=torch.bfloat16, device=dev) for _ in range(n_sets)]
    qws = torch.empty(max(1, ops.quantize_act_workspace_bytes(M, K, R), ops.quantize_act_workspace_bytes(M, F_out, R)),
                      dtype=torch.uint8, device=dev)

    def fused(i):
        a, b = sets13[i], sets2[i]
        ops.quantize_act(a["x"], a["layer"].smooth, a["layer"].proj_down, qact=q13[i], lora_act=l13[i], packed=True,
                         workspace=qws)
        ops.gemm_w4a4_gated_quant(q13[i], l13[i], a["layer"], M, b["layer"].smooth, h=hs[i], next_qact=q2[i])
        ops.lowrank_down(hs[i], b["layer"].proj_down, lora_act=l2[i], workspace=qws)
        ops.gemm_w4a4(q2[i], None, l2[i], b["layer"], y=b["y"], M=M)

    def gated_quant_gemm(i):
        a, b = sets13[i], sets2[i]
        ops.gemm_w4a4_gated_quant(q13[i], l13[i], a["layer"], M, b["layer"].smooth, h=hs[i], next_qact=q2[i])

    def w2_down(i):
        ops.lowrank_down(hs[i], sets2[i]["layer"].proj_down, lora_act=l2[i], workspace=qws)

    kw = max(1, args.warmup // 2)
    fused_ms = time_loop(fused, n_sets, max(10, args.kernel_iters // 4), kw, stream)
    gq_ms = time_loop(gated_quant_gemm, n_sets, max(10, args.kernel_iters // 4), kw, stream)
    w2d_ms = time_loop(w2_down, n_sets, args.kernel_iters, kw, stream)
    gated_ms = time_loop(gated_gemm, n_sets, args.kernel_iters, kw, stream)
    w2_ms = time_loop(w2_layer, n_sets, args.kernel_iters, kw, stream)
    unfused_ms = time_loop(unfused, n_sets, max(10, args.kernel_iters // 4), kw, stream)
    print(f"[bench] block with w2's input quantised in the gated epilogue: {fused_ms * 1e3:.1f} us "
          f"(that gated GEMM {gq_ms * 1e3:.1f} us, w2 down-projection alone {w2d_ms * 1e3:.1f} us)",
          file=sys.stderr, flush=True)
    gated_tflops = flops_gated_gemm / (gated_ms * 1e-3) / 1e12
    print(f"[bench] gated GEMM {gated_ms * 1e3:.1f} us ({gated_tflops:.1f} TFLOP/s), w2 layer {w2_ms * 1e3:.1f} us, "
          f"unfused block {unfused_ms * 1e3:.1f} us", file=sys.stderr, flush=True)
    result = {
        "metric": f"W4A4 SVDQuant FFN block (gated w1/w3 + w2) TFLOP/s at M={M},K={K},F={F_out}, 1 GPU",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f16",
        "data": "synthetic",
        "config": {
            "workload": f"{desc}: gated w1/w3 (one 2F-channel SVDQuant W4A4 layer, h = silu(gate) * up) "
                        f"then w2; M={M} K={K} F={F_out} N2={N2} R={R}",
            "cache": "warm" if args.warm else f"cold (rotating {n_sets} sets)",
            **({"gemm_tile_forced": args.gemm_tile} if args.gemm_tile else {}),
            "flop_per_step": flops_block,
        },
        "pct_mfma_peak": round(100.0 * tflops / PEAK_F16_MFMA_TFLOPS, 2),
        "roofline": {
            "kernel": "gemm_lds_kernel, gated (2F-channel GEMM + low-rank + silu(gate)*up epilogue)",
            "bound": "mfma",
            "achieved": round(gated_tflops, 2),
            "peak": PEAK_F16_MFMA_TFLOPS,
            "unit": "TFLOP/s",
            "frac": round(gated_tflops / PEAK_F16_MFMA_TFLOPS, 4),
            "traffic": None,
            "flop_per_launch": flops_gated_gemm,
            "avg_launch_us": round(gated_ms * 1e3, 2),
        },
        "w2_layer_us": round(w2_ms * 1e3, 2),
        "unfused_block_us": round(unfused_ms * 1e3, 2),
        "block_with_quantising_gate_us": round(fused_ms * 1e3, 2),
        "quantising_gated_gemm_us": round(gq_ms * 1e3, 2),
        "w2_down_projection_alone_us": round(w2d_ms * 1e3, 2),
    }
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle on the same block", file=sys.stderr, flush=True)
        t, threads = cpu_baseline_ffn(d13, d2, F_out)
        result["cpu_baseline"] = {"value": flops_block / t / 1e12, "unit": "TFLOP/s", "cores": threads,
                                  "kind": "oracle", "seconds_per_call": t,
                                  "sample": f"one FFN block call (M={M} K={K} F={F_out} N2={N2} R={R}); "
                                            f"{t:.2f} s; weight quantisation excluded (load time)"}
    print(json.dumps(result), flush=True)


def run_attn_block(args):
    """The attention half of a block with its linears in 8 bits: the norm that makes qkv's codes,
    qkv, rotary positions with the q/k norm (in place), attention, the out projection, and the
    gated norm that ends the half and starts the next."""
    import torch

    from bit_w4a4_quantized_quantize_amd import ops

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    cfg, desc = ATTN_BLOCKS[args.workload]
    M, K, H, text = cfg["M"], cfg["K"], cfg["H"], cfg["text"]
    D = K // H
    axes = (D // 4, 3 * D // 8, 3 * D // 8)   # text index (or frame), row, column
    bf = torch.bfloat16
    n_sets = 1 if args.warm else min(args.sets, 3)
    side = math.isqrt(M - text)
    j = torch.arange(M, device=dev)
    i = (j - text).clamp_min(0)
    pos = torch.stack([torch.where(j < text, j, text), i // side, i % side], 1).to(torch.int32)
    cu = torch.tensor([0, M], dtype=torch.int32, device=dev)
    sets = []
    for seed in range(n_sets):
        g = torch.Generator(device=dev).manual_seed(8100 + seed)
        rnd = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
        h = rnd(M, K)
        h[:, torch.randperm(K, generator=g, device=dev)[: K // 100]] *= 20.0
        qkv = torch.empty(M, 3 * K, dtype=bf, device=dev)
        q, k, v = (t.view(M, H, D) for t in qkv.split(K, 1))
        wqkv, wout = (rnd(3 * K, K) * 0.02).to(bf), (rnd(K, K) * 0.02).to(bf)
        e = dict(h=h.to(bf), qkv=qkv, q=q, k=k, v=v, wqkv=wqkv, wout=wout, qkv8=ops.quantize_int8(wqkv),
                 out8=ops.quantize_int8(wout), bias=(rnd(K) * 0.01).to(bf), pre=(1 + 0.1 * rnd(K)).to(bf),
                 post=(1 + 0.1 * rnd(K)).to(bf), pre2=(1 + 0.1 * rnd(K)).to(bf), gate=rnd(1, K).tanh().to(bf),
                 scale=(0.3 * rnd(1, K)).to(bf), scale2=(0.3 * rnd(1, K)).to(bf), qw=(1 + 0.1 * rnd(D)).to(bf),
                 kw=(1 + 0.1 * rnd(D)).to(bf), codes=torch.empty(M, K, dtype=torch.int8, device=dev),
                 cs=torch.empty(M, device=dev), o=torch.empty(M, H, D, dtype=bf, device=dev),
                 y=torch.empty(M, K, dtype=bf, device=dev), h2=torch.empty(M, K, dtype=bf, device=dev),
                 x2=torch.empty(M, K, dtype=bf, device=dev))
        e["ws"] = torch.empty(max(1, ops.gemm_int8_workspace_bytes(M, 3 * K, K),
                                  ops.linear_int8_workspace_bytes(M, K, K)), dtype=torch.uint8, device=dev)
        sets.append(e)

    parts = {
        "norm_to_codes": lambda e: ops.norm_gated_int8(e["h"], pre_weight=e["pre"], scale=e["scale"], codes=e["codes"],
                                                       scales=e["cs"]),
        "qkv_int8": lambda e: ops.gemm_int8(e["codes"], e["cs"], *e["qkv8"], y=e["qkv"], workspace=e["ws"]),
        "rope": lambda e: ops.rope_axes(e["q"], e["k"], pos, axes, theta=256.0, q_weight=e["qw"], k_weight=e["kw"],
                                        q_out=e["q"], k_out=e["k"]),
        "attention": lambda e: ops.attention_packed(e["q"], e["k"], e["v"], cu, out=e["o"]),
        "out_int8": lambda e: ops.linear_int8(e["o"].view(M, K), *e["out8"], bias=e["bias"], y=e["y"],
                                              workspace=e["ws"]),
        "norm_gated": lambda e: ops.norm_gated(e["h"], e["y"], post_weight=e["post"], gate=e["gate"],
                                               pre_weight=e["pre2"], scale=e["scale2"], h_out=e["h2"], x_out=e["x2"]),
    }

    def step(n):
        for part in parts.values():
            part(sets[n])

    flops = 2 * M * K * 4 * K + 4 * M * M * K
    ms_per_step, cond = timed(step, n_sets, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    tflops = flops / (ms_per_step * 1e-3) / 1e12
    kw = max(1, args.warmup // 2)
    iters = max(10, args.kernel_iters // 4)
    part_us = {name: round(time_loop(lambda n, f=f: f(sets[n]), n_sets, iters, kw, stream) * 1e3, 2)
               for name, f in parts.items()}
    # the same two linears kept in bf16, from the bf16 norm output
    x = ops.norm_gated(sets[0]["h"], pre_weight=sets[0]["pre"], scale=sets[0]["scale"])[1]
    part_us["qkv_bf16"] = round(time_loop(lambda n: ops.linear_bf16(x, sets[n]["wqkv"], y=sets[n]["qkv"]), n_sets,
                                          iters, kw, stream) * 1e3, 2)
    part_us["out_bf16"] = round(time_loop(lambda n: ops.linear_bf16(sets[n]["o"].view(M, K), sets[n]["wout"],
                                                                    y=sets[n]["y"]), n_sets, iters, kw, stream) * 1e3, 2)
    print(f"[bench] attention half-block: {ms_per_step * 1e3:.1f} us/step, {tflops:.1f} TFLOP/s "
          f"(conditioned {cond['conditioning_ms']:.1f} ms); parts in us: {part_us}", file=sys.stderr, flush=True)
    att = 4 * M * M * K / (part_us["attention"] * 1e-6) / 1e12
    print(json.dumps({
        "metric": f"attention half-block (norms, 8-bit qkv/out, rotary, attention) TFLOP/s at M={M},K={K},H={H}, 1 GPU",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int8 linears, bf16 attention",
        "data": "synthetic",
        "config": {"workload": f"{desc}: M={M} K={K} heads={H} of {D}, rotary axes {list(axes)}, full attention",
                   "cache": "warm" if args.warm else f"cold (rotating {n_sets} sets)", "flop_per_step": flops},
        "roofline": {"kernel": "attention_kernel", "bound": "mfma", "achieved": round(att, 2),
                     "peak": PEAK_F16_MFMA_TFLOPS, "unit": "TFLOP/s", "frac": round(att / PEAK_F16_MFMA_TFLOPS, 4),
                     "traffic": None, "flop_per_launch": 4 * M * M * K, "avg_launch_us": part_us["attention"]},
        "part_us": part_us,
    }), flush=True)


def sweep_build(dev, n_fwd, keep_prequant=False):
    """Weights of the sweep's 150 linears and fresh activations for n_fwd forwards, drawn on
    the device (torch's generator, seeded per layer / per (forward, layer)) with the
    distributions of the seeded host recipe: x ~ N(0,1) with 1% outlier channels x20 (fixed
    per layer), W ~ N(0, 0.02), proj ~ N(0, 0.02), bias ~ N(0, 0.01); the NVFP4 weights come
    from the library's own quantiser as in make_sets. With keep_prequant, each W4A4 entry
    also keeps "Wp", the bf16 weight W / (wtscale * wcscales) before quantisation (so that a
    check can quantise it independently)."""
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    bf = torch.bfloat16
    M, R = workloads.SWEEP_M, workloads.SWEEP_R
    layers = workloads.sweep_layers()
    built = []
    for L in layers:
        g = torch.Generator(device=dev).manual_seed(L["seed"])
        K, N = L["K"], L["N"]
        idx = torch.randperm(K, generator=g, device=dev)[: int(math.floor(0.01 * K))]
        e = dict(L, idx=idx)
        if L["precision"] == "bf16":
            e["W"] = (torch.randn(N, K, generator=g, device=dev) * 0.02).to(bf)
            e["b"] = (torch.randn(N, generator=g, device=dev) * 0.01).to(bf)
        else:
            xcal = torch.randn(M, K, generator=g, device=dev)
            xcal[:, idx] *= 20.0
            absmax = xcal.to(bf).float().abs().amax(0)
            smooth = (1.0 / absmax.clamp_min(1e-6).sqrt()).to(bf)
            del xcal
            W = torch.randn(N, K, generator=g, device=dev) * 0.02
            wc = (W.abs().amax(1).double() / (6.0 * 448.0)).to(bf)
            wt = torch.ones(1, dtype=bf, device=dev)
            Wp = (W / (wt.float() * wc.float())[:, None]).to(bf)
            del W
            qw, ws, _ = ops.quantize_act(Wp, torch.ones(K, dtype=bf, device=dev))
            if keep_prequant:
                e["Wp"] = Wp
            del Wp
            pd = (torch.randn(K, R, generator=g, device=dev) * 0.02).to(bf)
            pu = (torch.randn(N, R, generator=g, device=dev) * 0.02).to(bf)
            b = (torch.randn(N, generator=g, device=dev) * 0.01).to(bf)
            e["layer"] = ops.SVDQLinearWeights(N=N, K=K, weight=qw, wscales=ws, wcscales=wc, wtscale=wt,
                                               smooth=smooth, proj_down=pd, proj_up=pu, bias=b).packed()
        built.append(e)
    acts = []
    for f in range(n_fwd):
        row = []
        for li, L in enumerate(layers):
            g = torch.Generator(device=dev).manual_seed(workloads.sweep_activation_seed(f, li))
            x = torch.randn(M, L["K"], generator=g, device=dev)
            x[:, built[li]["idx"]] *= 20.0
            row.append(x.to(bf))
            del x
        acts.append(row)
    return built, acts


def sweep_flops(L, M, R):
    f = 2 * M * L["K"] * L["N"]
    return f + (2 * M * R * (L["K"] + L["N"]) if L["precision"] == "w4a4" else 0)


def cpu_baseline_sweep(M, R, layers):
    """The oracle on one bf16 layer and one W4A4 layer of the sweep, on a row sample, scaled to
    a whole forward by flop counts (an extrapolation: the oracle's per-flop rate at these
    shapes times the forward's flop count per precision)."""
    import numpy as np

    import workloads
    from oracle import svdq as S

    rows = 256
    d = workloads.make_bf16_linear(rows, 3840, 3840, kind="dit", seed=5001)
    t0 = time.perf_counter()
    S.linear_bf16(d["x"], d["W"], d["bias"])
    t_bf = time.perf_counter() - t0
    rate_bf = 2 * rows * 3840 * 3840 / t_bf
    d = workloads.make_linear(rows, 3840, 10240, R, kind="dit", seed=5002)
    qw, ws = S.quantize_weight(d["W"], d["wcscales"], d["wtscale"])   # load time, not timed
    t0 = time.perf_counter()
    S.linear_w4a4(d["x"], d["smooth"], qw, ws, d["wcscales"], d["wtscale"], d["proj_down"], d["proj_up"],
                  d["bias"])
    t_q = time.perf_counter() - t0
    rate_q = (2 * rows * 3840 * 10240 + 2 * rows * R * (3840 + 10240)) / t_q
    f_bf = sum(sweep_flops(L, M, R) for L in layers if L["precision"] == "bf16")
    f_q = sum(sweep_flops(L, M, R) for L in layers if L["precision"] == "w4a4")
    t_fwd = f_bf / rate_bf + f_q / rate_q
    try:
        from threadpoolctl import threadpool_info
        threads = max([i.get("num_threads", 1) for i in threadpool_info()] or [1])
    except Exception:
        threads = len(os.sched_getaffinity(0))
    del np
    return {"value": (f_bf + f_q) / t_fwd / 1e12, "unit": "TFLOP/s", "cores": int(threads), "kind": "oracle",
            "sample": f"{rows} rows of one bf16 out projection (3840->3840, {t_bf:.2f} s) and of one W4A4 "
                      f"w1 layer (3840->10240, R={R}, {t_q:.2f} s, weight quantisation excluded), "
                      f"extrapolated to one forward by flop count: {t_fwd:.1f} s per forward"}


def run_sweep(args):
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    M, R = workloads.SWEEP_M, workloads.SWEEP_R
    n_fwd = workloads.SWEEP_STEPS
    print(f"[bench] building the sweep: {workloads.SWEEP_BLOCKS} blocks, {n_fwd} forwards of fresh activations",
          file=sys.stderr, flush=True)
    t0 = time.perf_counter()
    built, acts = sweep_build(dev, n_fwd)
    layers = [{k: v for k, v in e.items() if k in ("block", "name", "K", "N", "precision")} for e in built]
    ys = {name: torch.empty((M, N), dtype=torch.bfloat16, device=dev) for name, _, N in workloads.SWEEP_LAYERS}
    ws_bytes = max(ops.linear_workspace_bytes(M, e["N"], e["K"], R) for e in built if e["precision"] == "w4a4")
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    print(f"[bench] built in {time.perf_counter() - t0:.1f} s; {torch.cuda.memory_allocated(dev) / 2**30:.1f} GiB "
          f"resident", file=sys.stderr, flush=True)
    flops_fwd = sum(sweep_flops(L, M, R) for L in layers)
    flops_bf = sum(sweep_flops(L, M, R) for L in layers if L["precision"] == "bf16")
    flops_q = flops_fwd - flops_bf

    def forward(f, which=("bf16", "w4a4")):
        for li, e in enumerate(built):
            if e["precision"] not in which:
                continue
            x = acts[f][li]
            if e["precision"] == "bf16":
                ops.linear_bf16(x, e["W"], e["b"], y=ys[e["name"]])
            else:
                ops.linear_w4a4(x, e["layer"], y=ys[e["name"]], workspace=ws)

    # eager, then one captured graph per forward (the launch sequence of a whole forward)
    for f in range(n_fwd):
        forward(f)
    torch.cuda.synchronize()
    graphs = []
    if not args.no_graph:
        for f in range(n_fwd):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                forward(f)
            graphs.append(g)
        torch.cuda.synchronize()

    def step(i):
        if graphs:
            graphs[i % n_fwd].replay()
        else:
            forward(i % n_fwd)

    t0 = time.perf_counter()
    ms_per_step, cond = timed(step, n_fwd, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    wall = time.perf_counter() - t0
    tflops = flops_fwd / (ms_per_step * 1e-3) / 1e12
    print(f"[bench] sweep ({'graph' if graphs else 'eager'}): {ms_per_step:.2f} ms per forward, {tflops:.1f} TFLOP/s "
          f"(wall {wall:.2f} s)", file=sys.stderr, flush=True)

    # split: the bf16 layers alone and the W4A4 layers alone (eager), and eager whole forwards
    def split_timed(fn, n):
        return timed(fn, n_fwd, n, stream, min_ms=10.0)[0]

    n_part = max(2, min(args.steps, n_fwd))
    bf_ms = split_timed(lambda i: forward(i % n_fwd, ("bf16",)), n_part)
    q_ms = split_timed(lambda i: forward(i % n_fwd, ("w4a4",)), n_part)
    eager_ms = split_timed(lambda i: forward(i % n_fwd), n_part)
    bf_tflops = flops_bf / (bf_ms * 1e-3) / 1e12
    q_tflops = flops_q / (q_ms * 1e-3) / 1e12
    print(f"[bench] bf16 layers {bf_ms:.2f} ms ({bf_tflops:.1f} TFLOP/s), W4A4 layers {q_ms:.2f} ms "
          f"({q_tflops:.1f} TFLOP/s), eager forward {eager_ms:.2f} ms", file=sys.stderr, flush=True)

    # the activation quantiser alone over the same tensors (the 60 W4A4 layers of a forward)
    qbuf = {}
    for e in built:
        if e["precision"] == "w4a4" and e["K"] not in qbuf:
            K = e["K"]
            qbuf[K] = (torch.empty(ops._lib.lib().svdq_packed_act_bytes(M, K), dtype=torch.uint8, device=dev),
                       torch.empty((M, R), dtype=torch.bfloat16, device=dev))
    qws = torch.empty(max(1, max(ops.quantize_act_workspace_bytes(M, K, R) for K in qbuf)), dtype=torch.uint8,
                      device=dev)

    def quant_fwd(f):
        for li, e in enumerate(built):
            if e["precision"] == "w4a4":
                qa, lo = qbuf[e["K"]]
                ops.quantize_act(acts[f][li], e["layer"].smooth, e["layer"].proj_down, qact=qa, lora_act=lo,
                                 packed=True, workspace=qws)

    quant_ms = split_timed(lambda i: quant_fwd(i % n_fwd), n_part)
    qbytes = sum(2 * M * e["K"] + 2 * e["K"] + 2 * e["K"] * R + M * e["K"] // 2 + M * e["K"] // 16 + 2 * M * R
                 for e in built if e["precision"] == "w4a4")
    quant_gbs = qbytes / (quant_ms * 1e-3) / 1e9
    print(f"[bench] activation quantiser over the forward's 60 W4A4 inputs: {quant_ms:.3f} ms "
          f"({quant_gbs:.0f} GB/s)", file=sys.stderr, flush=True)

    # single bf16 layer shapes, with torch's own bf16 linear (hipBLASLt) on the same operands as context
    shapes = {}
    for name, K, N in workloads.SWEEP_LAYERS:
        e = next(e for e in built if e["name"] == name and e["precision"] == "bf16")
        li = built.index(e)
        xs = [acts[f][li] for f in range(n_fwd)]
        ours = split_timed(lambda i: ops.linear_bf16(xs[i % n_fwd], e["W"], e["b"], y=ys[name]), 20)
        ref = split_timed(lambda i: torch.nn.functional.linear(xs[i % n_fwd], e["W"], e["b"]), 20)
        fl = 2 * M * K * N
        shapes[name] = {"K": K, "N": N, "us": round(ours * 1e3, 1), "TFLOPs": round(fl / (ours * 1e-3) / 1e12, 1),
                        "torch_linear_us": round(ref * 1e3, 1)}
    print(f"[bench] bf16 shapes: {shapes}", file=sys.stderr, flush=True)

    n_q = sum(1 for L in layers if L["precision"] == "w4a4")
    result = {
        "metric": f"DiT mixed-precision linear sweep TFLOP/s ({len(layers) - n_q} bf16 + {n_q} W4A4 NVFP4 linears "
                  f"per forward) at M={M}, 1 GPU",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 4),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16+f16",
        "data": "synthetic",
        "config": {
            "workload": SWEEPS[args.workload],
            "flop_per_step": flops_fwd,
            "flop_bf16": flops_bf,
            "flop_w4a4": flops_q,
            "launch": "one HIP graph per forward" if graphs else "eager",
            "cache": f"cold (fresh activations per (forward, layer), {n_fwd} forwards resident)",
        },
        "pct_mfma_peak": round(100.0 * tflops / PEAK_F16_MFMA_TFLOPS, 2),
        "roofline": {
            "kernel": "gemm_bf16_kernel (the bf16 layers: 55% of the forward's flops)",
            "bound": "mfma",
            "achieved": round(bf_tflops, 2),
            "peak": PEAK_F16_MFMA_TFLOPS,
            "unit": "TFLOP/s",
            "frac": round(bf_tflops / PEAK_F16_MFMA_TFLOPS, 4),
            "traffic": None,
            "flop_per_forward": flops_bf,
            "ms_per_forward": round(bf_ms, 4),
        },
        "w4a4_layers": {"ms_per_forward": round(q_ms, 4), "TFLOPs": round(q_tflops, 2)},
        "eager_ms_per_step": round(eager_ms, 4),
        "quant_kernel": {"ms_per_forward": round(quant_ms, 4), "hbm_bytes_per_forward": qbytes,
                         "achieved_GBps": round(quant_gbs, 1), "frac_of_hbm_peak": round(quant_gbs / PEAK_HBM_GBS, 4)},
        "bf16_shapes": shapes,
    }
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle on a sample of the sweep's layers", file=sys.stderr, flush=True)
        result["cpu_baseline"] = cpu_baseline_sweep(M, R, layers)
    print(json.dumps(result), flush=True)


def cpu_baseline_prep(W, sm, omega, iters, rows=1024):
    """The oracle's preparation: the randomized split on the whole weight (it needs all of
    it), the row-local residual and quantisation on `rows` rows, scaled to all rows."""
    from oracle import prep as P

    N = W.shape[0]
    t0 = time.perf_counter()
    pu, pd = P.lowrank_randomized(W, sm, omega, iters)
    t_split = time.perf_counter() - t0
    from oracle import formats as Fm
    pu_b, pd_b = Fm.f64_to_bf16(pu), Fm.f64_to_bf16(pd)
    t0 = time.perf_counter()
    E = P.residual(W[:rows], sm, pu_b[:rows], pd_b)
    P.quantize_residual(E)
    t_rows = time.perf_counter() - t0
    try:
        from threadpoolctl import threadpool_info
        threads = max([i.get("num_threads", 1) for i in threadpool_info()] or [1])
    except Exception:
        threads = len(os.sched_getaffinity(0))
    total = t_split + t_rows * N / rows
    return total, t_split, t_rows, int(threads)


def run_prep(args):
    import numpy as np
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    cfg = PREPS[args.workload]
    N, K, R, iters = cfg["N"], cfg["K"], cfg["R"], cfg["iters"]
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    W, sm, _ = workloads.make_prep_weight(N, K, seed=cfg["seed"])
    omega = workloads.make_omega(K, R, seed=cfg["seed"] + 1)

    def bf(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(dev)

    n_sets = 1 if args.warm else 3
    Wd = [bf(W) for _ in range(n_sets)]
    smd, omd = bf(sm), torch.from_numpy(omega).to(dev)
    ws = torch.empty(ops.prepare_workspace_bytes(N, K, R), dtype=torch.uint8, device=dev)
    steps, warmup = min(args.steps, 20), min(args.warmup, 5)

    def step(i):
        ops.prepare_weight(Wd[i % n_sets], smd, omd, iters=iters, workspace=ws)

    ms = time_loop(step, n_sets, steps, warmup, stream)
    ms0 = time_loop(lambda i: ops.prepare_weight(Wd[i % n_sets], smd, omd, iters=0, workspace=ws), n_sets,
                    steps, warmup, stream)
    # the residual stage alone (its own entry point, so it can be timed on the stream):
    # two fp64 passes of N*K*R fused multiply-adds (max |E| per row, then E / wcscales)
    lay = ops.prepare_weight(Wd[0], smd, omd, iters=iters, workspace=ws)
    res_ms = time_loop(lambda i: ops.prepare_residual(Wd[i % n_sets], smd, lay.proj_down, lay.proj_up,
                                                      workspace=ws), n_sets, steps, warmup, stream)
    flops_res = 2 * 2 * N * K * R
    res_tflops = flops_res / (res_ms * 1e-3) / 1e12
    print(f"[bench] preparation: {ms:.2f} ms per {N}x{K} weight (R={R}, {iters} power rounds; {ms0:.2f} ms "
          f"with none); residual stage {res_ms:.3f} ms ({res_tflops:.1f} TFLOP/s fp64)", file=sys.stderr, flush=True)
    result = {
        "metric": f"SVDQuant weight preparation time per weight at N={N},K={K},R={R}, 1 GPU",
        "value": round(ms, 3),
        "unit": "ms",
        "n_gpus": 1,
        "steps": steps,
        "warmup": warmup,
        "ms_per_step": round(ms, 4),
        "higher_is_better": False,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f32+f64",
        "data": "synthetic",
        "config": {"workload": cfg["desc"], "cache": "warm" if args.warm else f"rotating {n_sets} weights"},
        "roofline": {
            "kernel": "residual stage (svdq_prepare_residual: residual_kernel, fp64, then the quantiser); "
                      "most of the preparation's time is the Cholesky QR, then this stage and the fp32 "
                      "matrix-instruction products (profiles/prep_ffn_w1_1024_kernel_stats.txt)",
            "bound": "alu",
            "achieved": round(res_tflops, 2),
            "peak": PEAK_FP64_TFLOPS,
            "unit": "TFLOP/s",
            "frac": round(res_tflops / PEAK_FP64_TFLOPS, 4),
            "traffic": None,
            "flop_per_launch": flops_res,
            "avg_launch_us": round(res_ms * 1e3, 2),
        },
        "ms_iters0": round(ms0, 3),
        "ms_per_power_round": round((ms - ms0) / max(iters, 1), 3),
    }
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle on the same weight", file=sys.stderr, flush=True)
        total, t_split, t_rows, threads = cpu_baseline_prep(W, sm, omega, iters)
        result["cpu_baseline"] = {"value": round(total * 1e3, 1), "unit": "ms", "cores": threads, "kind": "oracle",
                                  "sample": f"randomized split on the whole weight ({t_split:.2f} s) plus residual "
                                            f"and quantisation of 1024 rows ({t_rows:.2f} s), scaled to {N} rows"}
    print(json.dumps(result), flush=True)


def run_mx(args):
    """The MXFP4 variant of a layer shape, beside the NVFP4 layer on the same inputs."""
    import torch

    from bit_w4a4_quantized_quantize_amd import ops

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    cfg, desc = workload_cfg(MX_VARIANTS[args.workload])
    M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]
    n_sets = 1 if args.warm else args.sets
    print(f"[bench] building {n_sets} input sets for M={M} K={K} N={N} R={R} (NVFP4, re-rounded to MXFP4)",
          file=sys.stderr, flush=True)
    d, sets = make_sets(cfg, n_sets, "canonical", dev)
    for st in sets:
        st["packed_layer"] = st["layer"].packed()
        st["mx_w"] = ops.reround_weight_mxfp4(st["layer"])
        st["mx_a"] = ops.quantize_act_mxfp4(st["x"], st["layer"].smooth)
        st["ws_mx"] = torch.empty(ops._lib.lib().svdq_linear_mxfp4_workspace_bytes(M, K, R), dtype=torch.uint8,
                                  device=dev)
        st["y_nv"] = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    torch.cuda.synchronize()
    flops_linear = 2 * M * N * K + 2 * M * R * (K + N)
    flops_gemm = 2 * M * N * K + 2 * M * N * R

    def step(i):
        st = sets[i]
        ops.linear_mxfp4(st["x"], st["layer"], st["mx_w"][0], st["mx_w"][1], y=st["y"], workspace=st["ws_mx"])

    ms, cond = timed(step, n_sets, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    tflops = flops_linear / (ms * 1e-3) / 1e12
    kw = max(1, args.warmup // 2)
    for st in sets:
        ops.quantize_act(st["x"], st["layer"].smooth, st["layer"].proj_down, qact=st["qact"],
                         ascales=st["ascales"], lora_act=st["lora"])
    torch.cuda.synchronize()
    gemm_ms = time_loop(lambda i: ops.gemm_mxfp4(sets[i]["mx_a"][0], sets[i]["mx_a"][1], sets[i]["lora"],
                                                 sets[i]["mx_w"][0], sets[i]["mx_w"][1], sets[i]["layer"], M,
                                                 y=sets[i]["y"]), n_sets, args.kernel_iters, kw, stream)
    nv_ms = time_loop(lambda i: ops.linear_w4a4(sets[i]["x"], sets[i]["packed_layer"], y=sets[i]["y_nv"],
                                                workspace=sets[i]["ws"]), n_sets, args.kernel_iters, kw, stream)
    gemm_tflops = flops_gemm / (gemm_ms * 1e-3) / 1e12
    # distance from the NVFP4 layer (both outputs from the library, same inputs)
    st = sets[0]
    ops.linear_mxfp4(st["x"], st["layer"], st["mx_w"][0], st["mx_w"][1], y=st["y"], workspace=st["ws_mx"])
    ops.linear_w4a4(st["x"], st["packed_layer"], y=st["y_nv"], workspace=st["ws"])
    torch.cuda.synchronize()
    dist = float(torch.linalg.vector_norm((st["y"].float() - st["y_nv"].float())) /
                 torch.linalg.vector_norm(st["y_nv"].float()))
    fp4_cal = calib_mfma(calib_tables(dev)["random_fp4_codes"], dev, stream, fmt=4)
    print(f"[bench] sustained scaled fp4 MFMA in this run: {fp4_cal}", file=sys.stderr, flush=True)
    print(f"[bench] MXFP4 layer {ms * 1e3:.1f} us ({tflops:.1f} TFLOP/s), its GEMM {gemm_ms * 1e3:.1f} us "
          f"({gemm_tflops:.1f} TFLOP/s); NVFP4 layer {nv_ms * 1e3:.1f} us; normwise distance {dist:.4f}",
          file=sys.stderr, flush=True)
    result = {
        "metric": f"MXFP4 variant of the SVDQuant linear, TFLOP/s at M={M},K={K},N={N}, 1 GPU (out of the "
                  f"NVFP4 tolerance: a speed point)",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "fp4",
        "data": "synthetic",
        "config": {"workload": f"{desc}, both operands re-rounded to MXFP4 (E2M1, E8M0 per 32 K); "
                               f"M={M} K={K} N={N} R={R}",
                   "cache": "warm" if args.warm else f"cold (rotating {n_sets} sets)",
                   **({"gemm_tile_forced": args.gemm_tile} if args.gemm_tile else {}),
                   "flop_per_step": flops_linear},
        "roofline": {
            "kernel": "gemm_mx_kernel (scaled FP4 matrix instruction + low-rank up-projection + epilogue)",
            "bound": "mfma",
            "achieved": round(gemm_tflops, 2),
            "peak": PEAK_FP4_MFMA_TFLOPS,
            "unit": "TFLOP/s",
            "frac": round(gemm_tflops / PEAK_FP4_MFMA_TFLOPS, 4),
            "traffic": None,
            "flop_per_launch": flops_gemm,
            "avg_launch_us": round(gemm_ms * 1e3, 2),
            "practical_peak": fp4_cal["TFLOPs"],
            "frac_of_practical": round(gemm_tflops / fp4_cal["TFLOPs"], 4),
            "practical_peak_note": "sustained v_mfma_scale_f32_32x32x64_f8f6f4 on random fp4 operands at the "
                                   "GEMM's occupancy, measured in this run",
        },
        "calibration_fp4": fp4_cal,
        "nvfp4_layer_us": round(nv_ms * 1e3, 2),
        "speedup_vs_nvfp4": round(nv_ms / ms, 3),
        "normwise_distance_from_nvfp4": round(dist, 5),
    }
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle on the variant layer", file=sys.stderr, flush=True)
        from oracle import mx as Xo
        from oracle import svdq as So
        qw, wsc = So.quantize_weight(d["W"], d["wcscales"], d["wtscale"])
        rows = 512
        t0 = time.perf_counter()
        Xo.linear_mxfp4(d["x"][:rows], d["smooth"], qw, wsc, d["wcscales"], d["wtscale"], d["proj_down"],
                        d["proj_up"], d["bias"])
        t = time.perf_counter() - t0
        fl = 2 * rows * N * K + 2 * rows * R * (K + N)
        try:
            from threadpoolctl import threadpool_info
            threads = max([i.get("num_threads", 1) for i in threadpool_info()] or [1])
        except Exception:
            threads = len(os.sched_getaffinity(0))
        result["cpu_baseline"] = {"value": fl / t / 1e12, "unit": "TFLOP/s", "cores": int(threads), "kind": "oracle",
                                  "sample": f"{rows} of the {M} rows ({t:.2f} s, including the weight re-round)"}
    print(json.dumps(result), flush=True)


def main():
    args = parse()
    if args.gemm_tile:
        from bit_w4a4_quantized_quantize_amd import ops
        ops.set_gemm_tile(args.gemm_tile)
        print(f"[bench] W4A4 GEMM tile shape forced to {args.gemm_tile} "
              f"({ {1: '256x320', 2: '256x256', 3: '128x320', 4: '128x160'}[args.gemm_tile] })",
              file=sys.stderr, flush=True)
    if args.workload in ORACLE_TIMES:
        return run_oracle_times(args)
    if args.workload in STATIC_VARIANTS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_static(args)
    if args.workload in CALIBS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_calib(args)
    if args.workload in MX_VARIANTS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_mx(args)
    if args.workload in PREPS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_prep(args)
    if args.workload in SWEEPS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_sweep(args)
    if args.workload in ATTN_BLOCKS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_attn_block(args)
    if args.workload in FFN_BLOCKS:
        if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
            print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
            sys.exit(2)
        return run_ffn_block(args)
    if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) > 1:
        print(json.dumps({"error": "this benchmark runs on exactly one GPU; the layer's multi-GPU "
                                   "sharding is described in the design notes but not built"}))
        print("bench.py: --gpus must be 1 (single-GPU build)", file=sys.stderr)
        sys.exit(2)

    import numpy as np
    import torch

    import workloads
    from bit_w4a4_quantized_quantize_amd import ops

    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    stream = torch.cuda.current_stream(dev)
    cfg, desc = workload_cfg(args.workload)
    M, K, N, R = cfg["M"], cfg["K"], cfg["N"], cfg["R"]
    n_sets = 1 if args.warm else args.sets
    print(f"[bench] building {n_sets} input sets for M={M} K={K} N={N} R={R} ({args.layout})",
          file=sys.stderr, flush=True)
    d, sets = make_sets(cfg, n_sets, args.layout, dev)
    torch.cuda.synchronize()

    flops_linear = 2 * M * N * K + 2 * M * R * (K + N)
    flops_gemm = 2 * M * N * K + 2 * M * N * R

    def step(i):
        s = sets[i]
        ops.linear_w4a4(s["x"], s["layer"], y=s["y"], workspace=s["ws"])

    # ---- headline: exactly K steps, synchronised on both sides ----
    # The chip is conditioned by time first (its clock settles over some milliseconds
    # of matrix work), then the W warm-up steps run, then the host synchronises; about
    # 1 ms of untimed steps is queued ahead of the start event so the timed steps begin
    # on a busy device rather than after the host's launch latency.
    t0 = time.perf_counter()
    ms_per_step, cond = timed(step, n_sets, args.steps, stream, warmup=args.warmup, min_ms=args.condition_ms)
    wall = time.perf_counter() - t0
    tflops = flops_linear / (ms_per_step * 1e-3) / 1e12
    print(f"[bench] linear: {ms_per_step * 1e3:.1f} us/step, {tflops:.1f} TFLOP/s "
          f"(conditioned {cond['conditioning_ms']:.1f} ms over {cond['conditioning_calls']} calls; "
          f"last windows {cond['conditioning_windows_us']} us/step; wall {wall:.2f} s)", file=sys.stderr, flush=True)

    # the per-step distribution (a separate pass with an event between steps) and the warm-cache
    # step (one set, the same buffers every call)
    step_dist = step_percentiles(step, n_sets, args.steps, stream)
    warm_ms = time_loop(step, 1, args.kernel_iters, max(1, args.warmup // 2), stream)
    print(f"[bench] per-step p10/p50/p90 {step_dist['p10']}/{step_dist['p50']}/{step_dist['p90']} us; "
          f"warm (one set) {warm_ms * 1e3:.1f} us/step", file=sys.stderr, flush=True)

    # ---- per-kernel timings, same stream and rotation, the kernels the step runs ----
    packed = args.layout == "packed"

    # as in the layer step: packed activations (with either weight layout), and the layer's
    # workspace (at least the quantiser's partial sums) passed so that no call allocates
    def quant_down(i):
        s = sets[i]
        ops.quantize_act(s["x"], s["layer"].smooth, s["layer"].proj_down, qact=s["qpk"],
                         lora_act=s["lora"], packed=True, workspace=s["ws"])

    for i in range(n_sets):
        quant_down(i)
    torch.cuda.synchronize()

    def gemm(i):
        s = sets[i]
        ops.gemm_w4a4(s["qpk"], None, s["lora"], s["layer"], y=s["y"], M=M)

    def quant(i):
        s = sets[i]
        ops.quantize_act(s["x"], s["layer"].smooth, None, qact=s["qact"], ascales=s["ascales"])

    kw = max(1, args.warmup // 2)
    gemm_ms = time_loop(gemm, n_sets, args.kernel_iters, kw, stream)
    warm_gemm_ms = time_loop(gemm, 1, args.kernel_iters, kw, stream)
    quant_ms = time_loop(quant, n_sets, args.kernel_iters, kw, stream)
    qd_ms = time_loop(quant_down, n_sets, args.kernel_iters, kw, stream)
    gemm_tflops = flops_gemm / (gemm_ms * 1e-3) / 1e12
    quant_bytes_a1 = M * K * 2 + K * 2 + M * K // 2 + (K // 16) * M
    quant_bytes_fused = quant_bytes_a1 + 2 * K * R + 2 * M * R
    quant_gbs = quant_bytes_a1 / (quant_ms * 1e-3) / 1e9
    print(f"[bench] gemm kernel {gemm_ms * 1e3:.1f} us ({gemm_tflops:.1f} TFLOP/s), quant {quant_ms * 1e3:.2f} us "
          f"({quant_gbs:.0f} GB/s), quant+down {qd_ms * 1e3:.2f} us", file=sys.stderr, flush=True)

    # practical ceilings on this device, measured now: sustained f16 MFMA on exact NVFP4
    # operand values and on random f16 bits, and a streaming device copy
    calib = calibration(dev, stream, quick=True)
    practical = calib["mfma_f16_32x32x16"]["nvfp4_values"]["TFLOPs"]
    copy_gbs = calib["copy_1GiB"]["GBps"]
    print(f"[bench] calibration: {calib}", file=sys.stderr, flush=True)

    # the committed counters were taken on the packed-path GEMM at the headline workload
    traffic = read_traffic() if packed and args.workload == DEFAULT_WORKLOAD else None
    result = {
        "metric": METRIC if args.workload == DEFAULT_WORKLOAD else
                  f"W4A4 SVDQuant linear TFLOP/s and % MFMA peak at M={M},K={K},N={N}, 1 GPU",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms_per_step, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "f16",
        "data": "synthetic",
        "config": {
            "workload": f"{desc}: SVDQuant W4A4 NVFP4 linear, M={M} K={K} N={N} R={R}",
            "weight_layout": args.layout,
            "cache": "warm" if args.warm else f"cold (rotating {n_sets} sets)",
            **({"gemm_tile_forced": args.gemm_tile} if args.gemm_tile else {}),
            "flop_per_step": flops_linear,
            "arithmetic": "exact NVFP4 dequant to f16, f16 MFMA with fp32 accumulation; "
                          "low-rank in bf16 MFMA; quantisation in fp32",
        },
        "pct_mfma_peak": round(100.0 * tflops / PEAK_F16_MFMA_TFLOPS, 2),
        "roofline": {
            "kernel": "gemm_lds_kernel (scaled GEMM + low-rank up-projection + epilogue)"
                      + ("" if args.layout == "packed" else ", reading the canonical weight layout"),
            "bound": "mfma",
            "achieved": round(gemm_tflops, 2),
            "peak": PEAK_F16_MFMA_TFLOPS,
            "unit": "TFLOP/s",
            "frac": round(gemm_tflops / PEAK_F16_MFMA_TFLOPS, 4),
            "traffic": traffic,
            "flop_per_launch": flops_gemm,
            "avg_launch_us": round(gemm_ms * 1e3, 2),
            "practical_peak": practical,
            "frac_of_practical": round(gemm_tflops / practical, 4),
            "practical_peak_note": "sustained v_mfma_f32_32x32x16_f16 at the GEMM's occupancy on exact NVFP4 "
                                   "operand values, measured in this run (the chip power-limits its clock "
                                   "under sustained matrix work)",
        },
        "quant_kernel": {
            "avg_launch_us": round(quant_ms * 1e3, 3),
            "hbm_bytes_per_launch": quant_bytes_a1,
            "achieved_GBps": round(quant_gbs, 1),
            "frac_of_hbm_peak": round(quant_gbs / PEAK_HBM_GBS, 4),
            "practical_copy_GBps": copy_gbs,
            "frac_of_practical_copy": round(quant_gbs / copy_gbs, 4),
            "kernel": "quant_act_kernel (activation quantisation alone, canonical output)",
            "fused_with_down_projection_us": round(qd_ms * 1e3, 3),
            "fused_hbm_bytes_per_launch": quant_bytes_fused,
            "fused_achieved_GBps": round(quant_bytes_fused / (qd_ms * 1e-3) / 1e9, 1),
        },
        "conditioning": cond,
        "step_us": step_dist,
        "warm_step_us": round(warm_ms * 1e3, 2),
        "warm_gemm_us": round(warm_gemm_ms * 1e3, 2),
        "calibration": calib,
        "device": device_info(dev),
    }
    if args.copy_calibration:
        # a plain 512 MiB streaming copy, to calibrate the profiler's HBM byte counters
        L = ops._lib.lib()
        src = torch.empty(512 << 20, dtype=torch.uint8, device=dev)
        dst = torch.empty_like(src)
        for _ in range(3):
            ops._lib.check("svdq_calib_copy", L.svdq_calib_copy(src.data_ptr(), dst.data_ptr(), src.numel(),
                                                                stream.cuda_stream))
        torch.cuda.synchronize()
        del src, dst
    if not args.no_cpu_baseline:
        print("[bench] timing the CPU oracle on the same workload", file=sys.stderr, flush=True)
        result["cpu_baseline"] = cpu_baseline(d, cfg)
    print(json.dumps(result), flush=True)


if __name__ == "__main__":
    main()
