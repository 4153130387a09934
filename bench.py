"""Benchmark: GPTQ layer quantization throughput on one MI355X.

One step is one full pass of the layer quantizer over one linear layer with its
calibration activations already resident in HBM: H = 0; H += 2 X^T X
(gptq_accumulate_hessian); damping, factor and the 128-column quantize loop
with trailing updates (gptq_quantize_layer); packing (gptq_pack).

Default workload: one Llama-2-7B q_proj-shaped layer, W 4096x4096 bf16
~N(0, 0.02^2), X 262144 tokens x 4096 bf16 Student-t(4) with 41 outlier
channels x20, 4-bit asymmetric, groupsize 128, block 128, damp 0.01.

Prints one JSON line.  Stage times come from HIP events on the stream the
library launches on (PyTorch's current stream).
"""

from __future__ import annotations

import argparse
import hashlib
import json
import os
import sys
import time

import numpy as np

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "GPTQ layers/sec + TFLOP/s (4096×4096 & 11008×4096, 4-bit g128) vs MFMA peak"
PEAK_BF16_TFLOPS = 2500.0
PEAK_F32_TFLOPS = 157.3
PEAK_HBM_GBS = 8000.0

# HBM bytes per Hessian accumulation call (k_syrk_bf16 and k_syrk_reduce together), from two
# rocprofv3 counter passes (FETCH_SIZE, WRITE_SIZE) scaled by the reading of a plain 1 GiB copy;
# the summary with the commands is profiles/hbm_counters_q_proj_4096x4096_262144tok.md.  Valid
# only for the kernel sources they were taken on (k_hessian.hip and the work decomposition it
# includes, syrk_plan.h): different sources report null.
SYRK_TRAFFIC = {"sources_sha256": "8952fbf7191d791ea96c51eeffa863712a8eb695bbba17f28e1574468b8b3e5f",
                "workload": "q_proj_4096", "tokens": 262144,
                "fetch_bytes": 9207576928.4, "write_bytes": 492600896.0}
SYRK_SOURCES = ("k_hessian.hip", "syrk_plan.h")


def syrk_sources_sha256():
    h = hashlib.sha256()
    for name in SYRK_SOURCES:
        with open(os.path.join(ROOT, "post_weight_quantization_03_amd", "csrc", name), "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def syrk_traffic(workload, tokens):
    t = SYRK_TRAFFIC
    if syrk_sources_sha256() != t["sources_sha256"] or workload != t["workload"] or tokens != t["tokens"]:
        return None
    return t["fetch_bytes"] + t["write_bytes"]


def parse():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--warmup", type=int, default=2)
    ap.add_argument("--workload", default="q_proj_4096")
    ap.add_argument("--tokens", type=int, default=None, help="override the calibration token count")
    ap.add_argument("--layer", type=int, default=0, help="which linear layer of the workload (default the first)")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--cpu-tokens", type=int, default=16384, help="tokens in the oracle's Hessian sample")
    ap.add_argument("--cpu-rows", type=int, default=512, help="rows in the oracle's quantize sample")
    ap.add_argument("--no-extras", action="store_true",
                    help="skip the measurements outside the timed step (GEMV, rotation, error-propagation correction)")
    ap.add_argument("--whole", action="store_true",
                    help="one step = every Hessian and every linear layer of the workload, in order, "
                         "with all inputs resident (layers that share a Hessian reuse its factor)")
    ap.add_argument("--calib-copy", action="store_true",
                    help="also run one plain 1 GiB device copy (HBM counter calibration under rocprofv3)")
    ap.add_argument("--cpu-full", action="store_true",
                    help="time the oracle over the whole layer (every token, every row) instead of a sample")
    ap.add_argument("--no-second", action="store_true",
                    help="skip the metric's second shape (11008x4096, 4-bit g128) on the default workload")
    ap.add_argument("--trace", action="store_true",
                    help="instead of the bench line: one pass of the layer on libgptq_trace.so, printing the "
                         "phase timestamps of the column loop and the factor's chain (medians, us), and one "
                         "call of the batch product (5120x25600, 8 fp32 vectors) with its workgroups' phases")
    return ap.parse_args()


def algorithmic(rows, cols, tokens, bits):
    """Algorithmic work of one step: the symmetric Hessian N n(n+1) flops, the factor 2n^3/3,
    the quantize loop rows*cols^2 of which the trailing update rows*cols*(cols-128)."""
    hess = tokens * cols * (cols + 1)
    factor = 2.0 * cols ** 3 / 3.0
    quant = float(rows) * cols * cols
    trailing = float(rows) * cols * max(cols - 128, 0)
    x_bytes = 2.0 * tokens * cols
    return {"hessian_flop": float(hess), "factor_flop": factor, "quantize_flop": quant,
            "trailing_flop": trailing, "x_bytes": x_bytes,
            "total_flop": float(hess) + factor + quant}


def cpu_info():
    """The host the oracle runs on: core counts, CPU model and the BLAS libraries in use."""
    model = "unknown"
    try:
        with open("/proc/cpuinfo") as f:
            model = next((l.split(":", 1)[1].strip() for l in f if l.startswith("model name")), model)
    except OSError:  # pragma: no cover
        pass
    blas = []
    try:
        from threadpoolctl import threadpool_info
        blas = [{k: d.get(k) for k in ("internal_api", "version", "num_threads", "architecture")}
                for d in threadpool_info() if d.get("user_api") == "blas"]
    except Exception:  # pragma: no cover
        pass
    try:
        affinity = len(os.sched_getaffinity(0))
    except AttributeError:  # pragma: no cover
        affinity = os.cpu_count()
    return {"cpu_count": os.cpu_count(), "affinity": affinity, "cpu_model": model, "blas": blas}


def cpu_baseline(W, acts, rows, cols, tokens, bits, args, x_bf16=True, w_bf16=True):
    """The oracle on the host cores: the Hessian over a token sample (or every token), the damped
    factor of the full layer, and the lazy-batch GPTQ loop over a row sample (or every row), each
    timed on its own and scaled to one full layer."""
    from oracle import damp_ref, factor_ref, gptq_from_factor, hessian_ref
    from post_weight_quantization_03_amd import synth
    info = cpu_info()
    threads = max([b["num_threads"] or 1 for b in info["blas"]] or [os.cpu_count() or 1])
    nt = tokens if args.cpu_full else min(args.cpu_tokens, tokens)
    nr = rows if args.cpu_full else min(args.cpu_rows, rows)

    def chunks():
        for t0 in range(0, nt, 16384):
            blk = acts.block(t0, min(16384, nt - t0))
            yield synth.bf16_to_f32(blk) if x_bf16 else blk

    t0 = time.perf_counter()
    H = hessian_ref(chunks(), cols)
    t_h = time.perf_counter() - t0
    H *= tokens / nt  # a same-law stand-in for the full-token Hessian when sampled
    Ws = (synth.bf16_to_f32(W[:nr]) if w_bf16 else W[:nr]).astype(np.float64)
    t0 = time.perf_counter()
    Hd, Ws, _, _ = damp_ref(H, Ws, 0.01)
    U = factor_ref(Hd)
    t_f = time.perf_counter() - t0
    del H, Hd
    t0 = time.perf_counter()
    gptq_from_factor(Ws, U, bits, 128, blocksize=128)
    t_q = time.perf_counter() - t0
    est = t_h * (tokens / nt) + t_f + t_q * (rows / nr)
    if args.cpu_full:
        sample = (f"fp64 NumPy oracle over the whole layer: Hessian over all {tokens} tokens, {cols}x{cols} "
                  f"factor, lazy-batch GPTQ loop over all {rows} rows; measured {t_h:.2f}s + {t_f:.2f}s + "
                  f"{t_q:.2f}s")
    else:
        sample = (f"fp64 NumPy oracle: Hessian over {nt} of {tokens} tokens (x{tokens / nt:g}), "
                  f"full {cols}x{cols} factor, lazy-batch GPTQ loop over {nr} of {rows} rows "
                  f"(x{rows / nr:g}); measured {t_h:.2f}s + {t_f:.2f}s + {t_q:.2f}s")
    return {"value": 1.0 / est, "unit": "layers/s", "cores": int(threads), "kind": "oracle", "sample": sample,
            "seconds_full_layer": est, "measured_in_full": bool(args.cpu_full),
            "stage_seconds": {"hessian": t_h, "factor": t_f, "quantize_loop": t_q}, "host": info}


def gemv_measure(g, torch, packed, scales, zeros, rows, cols, bits, groupsize, dev, rounds=4):
    """y = W^ x over this step's packed layer (gptq_dequant_gemv), outside the timed step.

    Each launch reads its own copy of the packed codes, scales and zeros, and the
    copies together exceed the 256 MB last-level cache, so every launch reads its
    weights from HBM as a model's layers would.  The launches are queued behind a
    short device-side sleep, so the HIP events around them time back-to-back
    kernels rather than the host's launch rate.
    """
    import ctypes
    G = scales.shape[1]
    alg_bytes = rows * cols * bits / 8 + rows * G * 5 + cols * 4 + rows * 4
    copies = int(max(2, -(-(512 << 20) // int(alg_bytes))))
    bufs = [(packed.clone(), scales.clone(), zeros.clone()) for _ in range(copies)]
    x = torch.randn(cols, dtype=torch.float32, device=dev, generator=torch.Generator(dev).manual_seed(1))
    y = torch.empty(rows, dtype=torch.float32, device=dev)
    for p, s_, z in bufs:  # checked binding once per buffer set
        g.gptq_dequant_gemv(p, s_, z, bits, groupsize, x, y)
    fn = g.lib().gptq_dequant_gemv
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    calls = [(ctypes.c_void_p(p.data_ptr()), ctypes.c_void_p(s_.data_ptr()), ctypes.c_void_p(z.data_ptr()), rows,
              cols, bits, groupsize, ctypes.c_void_p(x.data_ptr()), g.GPTQ_F32, ctypes.c_void_p(y.data_ptr()),
              stream)
             for p, s_, z in bufs]
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda._sleep(50_000_000)
    e0.record()
    for _ in range(rounds):
        for a in calls:
            st = fn(*a)
            if st:
                raise RuntimeError(f"gptq_dequant_gemv: status {st}")
    e1.record()
    torch.cuda.synchronize()
    us = e0.elapsed_time(e1) * 1e3 / (rounds * copies)
    gbs = alg_bytes / (us * 1e-6) / 1e9
    # the same weights against a batch of 8 vectors (gptq_dequant_gemm)
    B = 8
    Xb = torch.randn(B, cols, dtype=torch.float32, device=dev, generator=torch.Generator(dev).manual_seed(2))
    Yb = torch.empty(B, rows, dtype=torch.float32, device=dev)
    fb = g.lib().gptq_dequant_gemm
    wsb = g.gptq_dequant_gemm_workspace_bytes(rows, cols, bits, groupsize, B)
    wsp = torch.empty(max(wsb, 256), dtype=torch.uint8, device=dev)
    bcalls = [(ctypes.c_void_p(p.data_ptr()), ctypes.c_void_p(s_.data_ptr()), ctypes.c_void_p(z.data_ptr()), rows,
               cols, bits, groupsize, ctypes.c_void_p(Xb.data_ptr()), g.GPTQ_F32, cols, B,
               ctypes.c_void_p(Yb.data_ptr()), rows, ctypes.c_void_p(wsp.data_ptr()), wsb, stream)
              for p, s_, z in bufs]
    for a in bcalls:
        if fb(*a):
            raise RuntimeError("gptq_dequant_gemm failed")
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    e0.record()
    for _ in range(rounds):
        for a in bcalls:
            fb(*a)
    e1.record()
    torch.cuda.synchronize()
    us_b = e0.elapsed_time(e1) * 1e3 / (rounds * copies)
    bytes_b = alg_bytes + (B - 1) * (cols + rows) * 4
    return {"kernel": "k_dequant_gemv", "shape": [rows, cols], "bits": bits, "groupsize": groupsize,
            "us_per_launch": us, "algorithmic_bytes": alg_bytes, "achieved_GBs": gbs, "peak_GBs": PEAK_HBM_GBS,
            "frac": gbs / PEAK_HBM_GBS, "weight_copies": copies,
            "batch8": {"kernel": ("k_dequant_mma" + (" + k_mma_reduce" if wsb else "")
                                  if groupsize == -1 or groupsize % 128 == 0 else "k_dequant_gemm"),
                       "us_per_launch": us_b, "algorithmic_bytes": bytes_b,
                       "achieved_GBs": bytes_b / (us_b * 1e-6) / 1e9,
                       "frac": bytes_b / (us_b * 1e-6) / 1e9 / PEAK_HBM_GBS, "us_per_vector": us_b / B}}


def gemv_shapes_measure(g, torch, dev, bits=4, groupsize=128):
    """The dequantizing GEMV and the batch-8 GEMM on the other layer shapes of the workloads
    (Llama-2-7B gate/up 11008x4096 and down 4096x11008, Qwen3-32B down 5120x25600), 4-bit g128,
    over seeded random packed codes, scales in [0.005, 0.02] and zero points (the kernels' work
    does not depend on the values), timed as gemv_measure times the step's own layer."""
    out = {}
    gen = torch.Generator(dev).manual_seed(5)
    for rows, cols in ((11008, 4096), (4096, 11008), (5120, 25600)):
        G = -(-cols // groupsize)
        packed = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols * bits // 32), dtype=torch.int32, device=dev,
                               generator=gen)
        scales = 0.005 + 0.015 * torch.rand((rows, G), device=dev, generator=gen)
        zeros = torch.randint(0, 2 ** bits, (rows, G), dtype=torch.uint8, device=dev, generator=gen)
        r = gemv_measure(g, torch, packed, scales, zeros, rows, cols, bits, groupsize, dev)
        out[f"{rows}x{cols}"] = {k: r[k] for k in ("us_per_launch", "algorithmic_bytes", "achieved_GBs", "frac",
                                                   "weight_copies", "batch8")}
        del packed, scales, zeros, r
        torch.cuda.empty_cache()
    return out


def hadamard_measure(g, torch, Wd, n, dev, copies=6, rounds=3):
    """The fixed Hadamard rotation (block n) on this layer, outside the timed step:
    W' = W Q from bf16 W (gptq_hadamard_rows) and H' = Q^T H Q in place
    (gptq_hadamard_hessian), each over several copies larger than the last-level
    cache together, queued behind a short device sleep and timed with HIP events."""
    import ctypes
    rows = Wd.shape[0]
    block = n & -n
    while block > 4096:
        block //= 2
    gen = torch.Generator(dev).manual_seed(2)
    signs = torch.where(torch.rand(n, device=dev, generator=gen) < 0.5, -1.0, 1.0).float()
    Ws = [Wd.clone() for _ in range(copies)]
    Wo = [torch.empty((rows, n), dtype=torch.float32, device=dev) for _ in range(copies)]
    Hs = []
    for _ in range(copies):
        a = torch.randn(n, n, device=dev, generator=gen)
        Hs.append(a + a.T)
    L = g.lib()
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    sp = ctypes.c_void_p(signs.data_ptr())

    def timed(fn):
        fn()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(20_000_000)
        e0.record()
        for _ in range(rounds):
            fn()
        e1.record()
        torch.cuda.synchronize()
        return e0.elapsed_time(e1) * 1e3 / (rounds * copies)

    def rot_w():
        for a, b in zip(Ws, Wo):
            if L.gptq_hadamard_rows(ctypes.c_void_p(a.data_ptr()), g.GPTQ_BF16, n, ctypes.c_void_p(b.data_ptr()), n,
                                    rows, n, sp, block, st):
                raise RuntimeError("gptq_hadamard_rows failed")

    def rot_h():
        for h in Hs:
            if L.gptq_hadamard_hessian(ctypes.c_void_p(h.data_ptr()), n, sp, block, st):
                raise RuntimeError("gptq_hadamard_hessian failed")

    us_w, us_h = timed(rot_w), timed(rot_h)
    bytes_w = rows * n * (2 + 4) + n * 4
    bytes_h = 2 * n * n * 4 + n * 4
    return {"kernels": "k_hadamard_rows, k_tile_pairs", "block": block,
            "weights_us": us_w, "weights_algorithmic_bytes": bytes_w, "weights_GBs": bytes_w / us_w / 1e3,
            "weights_frac": bytes_w / us_w / 1e3 / PEAK_HBM_GBS,
            "hessian_us": us_h, "hessian_algorithmic_bytes": bytes_h, "hessian_GBs": bytes_h / us_h / 1e3,
            "hessian_frac": bytes_h / us_h / 1e3 / PEAK_HBM_GBS}


def qep_measure(g, torch, Xd, Wd, n, dev):
    """The error-propagation correction on this layer, outside the timed step: the cross
    term C = 2 X^T X^ over all tokens (X^ = X + 5 % noise stands in for the quantized
    model's inputs) and the correction W' = W + alpha W (C - H) H_d^-1, which also leaves
    H factored for the quantizer.  HIP events around each call."""
    gen = torch.Generator(dev).manual_seed(3)
    Xq = torch.empty_like(Xd)
    for a in range(0, Xd.shape[0], 16384):  # bounded temporaries
        xs = Xd[a:a + 16384].float()
        Xq[a:a + 16384] = (xs + 0.05 * xs.std() * torch.randn(xs.shape, device=dev, generator=gen)).to(Xd.dtype)
    del xs
    H = torch.zeros((n, n), dtype=torch.float32, device=dev)
    C = torch.zeros((n, n), dtype=torch.float32, device=dev)
    ws_h = torch.empty(max(g.gptq_hessian_workspace_bytes(n, Xd.shape[0], g.GPTQ_BF16), 1), dtype=torch.uint8,
                       device=dev)
    ws_c = torch.empty(max(g.gptq_cross_workspace_bytes(n, Xd.shape[0], g.GPTQ_BF16), 1), dtype=torch.uint8,
                       device=dev)
    ws_q = torch.empty(g.gptq_qep_workspace_bytes(Wd.shape[0], n), dtype=torch.uint8, device=dev)
    Wout = torch.empty((Wd.shape[0], n), dtype=torch.float32, device=dev)
    dst = torch.zeros((1,), dtype=torch.int32, device=dev)
    times = {"cross": [], "correct": []}
    for rep in range(3):
        H.zero_()
        C.zero_()
        g.gptq_accumulate_hessian(H, Xq, workspace=ws_h)
        e = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        e[0].record()
        g.gptq_accumulate_cross(C, Xd, Xq, workspace=ws_c)
        e[1].record()
        g.gptq_qep_correct(Wd, C, H, 0.5, W_out=Wout, workspace=ws_q, d_status=dst)
        e[2].record()
        torch.cuda.synchronize()
        if rep:
            times["cross"].append(e[0].elapsed_time(e[1]))
            times["correct"].append(e[1].elapsed_time(e[2]))
    if int(dst.item()) != 0:
        raise SystemExit(f"qep correction status {int(dst.item())}")
    t_c = float(np.mean(times["cross"])) / 1e3
    t_q = float(np.mean(times["correct"])) / 1e3
    N = Xd.shape[0]
    flop_c = 2.0 * N * n * n
    return {"kernels": "k_syrk_bf16 cross mode + k_syrk_reduce (cross term); factor + k_gemm_f32 x3 (correction)",
            "tokens": N, "alpha": 0.5, "cross_ms": t_c * 1e3, "cross_tflops": flop_c / t_c / 1e12,
            "cross_frac_bf16_peak": flop_c / t_c / 1e12 / PEAK_BF16_TFLOPS,
            "correct_ms_incl_factor": t_q * 1e3}


def host_tensor(torch, a, bf16):
    """A generated host array as a torch tensor: bf16 bit patterns (uint16) or fp32."""
    return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16) if bf16 else torch.from_numpy(a)


def whole_workload(args, g, torch, wl, dev):
    """Time one pass over every layer of a workload: per Hessian, H = 0 and H += 2 X^T X;
    per linear, damping, factor and quantize loop (the first layer on a Hessian factors it,
    the others reuse the factor through GPTQ_H_IS_FACTOR) and packing.  Every Hessian's
    activations and every layer's weights are a tensor of their own, resident in HBM before
    the timed region; codes go to one scratch buffer per shape, scales, zeros and packed
    codes to buffers of their own per layer."""
    t0 = time.perf_counter()
    # one generated tensor per shape; every Hessian and every layer then gets a copy of its
    # own, rolled by a distinct offset along the tokens (activations) or rows (weights), so
    # no two calls read the same memory and the values keep the generator's law
    base_x, X = {}, {}
    for i, (name, acts) in enumerate(wl.hessians.items()):
        key = (acts.n, acts.tokens)
        if key not in base_x:
            Xd = torch.empty((acts.tokens, acts.n), dtype=torch.bfloat16 if acts.bf16 else torch.float32,
                             device=dev)
            for t, blk in zip(range(0, acts.tokens, acts.chunk), acts.chunks()):
                Xd[t:t + blk.shape[0]].copy_(host_tensor(torch, blk, acts.bf16))
            base_x[key] = Xd
            print(f"bench.py: activations {acts.tokens}x{acts.n} generated ({time.perf_counter() - t0:.0f} s)",
                  file=sys.stderr, flush=True)
        X[name] = torch.roll(base_x[key], shifts=(97 * i) % acts.tokens, dims=0)
    del base_x
    base_w, Ws = {}, []
    for i, lin in enumerate(wl.linears):
        key = (lin.rows, lin.cols)
        if key not in base_w:
            base_w[key] = host_tensor(torch, lin.weight(), lin.bf16).to(dev)
        Ws.append(torch.roll(base_w[key], shifts=(13 * i) % lin.rows, dims=0))
    del base_w
    torch.cuda.synchronize()
    print(f"bench.py: {len(X)} activation and {len(Ws)} weight tensors resident ({time.perf_counter() - t0:.0f} s)",
          file=sys.stderr, flush=True)
    gen_s = time.perf_counter() - t0

    Hbuf = {n: torch.zeros((n, n), dtype=torch.float32, device=dev) for n in {a.n for a in wl.hessians.values()}}
    codes = {(l.rows, l.cols): torch.empty((l.rows, l.cols), dtype=torch.uint8, device=dev) for l in wl.linears}
    params, outs = [], []
    ws_q_bytes = ws_h_bytes = 1
    for lin in wl.linears:
        p = g.Params(bits=lin.bits, groupsize=wl.groupsize, blocksize=wl.blocksize, damp=wl.damp)
        params.append(p)
        G = -(-lin.cols // wl.groupsize)
        outs.append((torch.empty((lin.rows, G), dtype=torch.float32, device=dev),
                     torch.empty((lin.rows, G), dtype=torch.uint8, device=dev),
                     torch.empty((lin.rows,), dtype=torch.float32, device=dev),
                     torch.empty((lin.rows, lin.cols * lin.bits // 32), dtype=torch.int32, device=dev)))
        ws_q_bytes = max(ws_q_bytes, g.gptq_quantize_workspace_bytes(lin.rows, lin.cols, p))
    for a in wl.hessians.values():
        ws_h_bytes = max(ws_h_bytes, g.gptq_hessian_workspace_bytes(a.n, a.tokens,
                                                                     g.GPTQ_BF16 if a.bf16 else g.GPTQ_F32))
    ws_h = torch.empty(ws_h_bytes, dtype=torch.uint8, device=dev)
    ws_q = torch.empty(ws_q_bytes, dtype=torch.uint8, device=dev)
    dstat = torch.zeros((1,), dtype=torch.int32, device=dev)
    kinds = {"hessian": [], "factor_and_quantize": [], "pack": []}

    def step(record):
        marks = []

        def mark(kind):
            if record:
                e = torch.cuda.Event(enable_timing=True)
                e.record()
                marks.append((kind, e))

        current = None
        for lin, W, p, (scales, zeros, loss, packed) in zip(wl.linears, Ws, params, outs):
            H = Hbuf[lin.cols]
            shared = lin.hessian == current
            if not shared:
                H.zero_()
                mark(None)
                g.gptq_accumulate_hessian(H, X[lin.hessian], workspace=ws_h)
                mark("hessian")
                current = lin.hessian
            q = p if not shared else g.Params(p.bits, p.groupsize, p.blocksize, p.damp, g.GPTQ_H_IS_FACTOR)
            c = codes[(lin.rows, lin.cols)]
            mark(None)
            g.gptq_quantize_layer(W, H, q, c, scales, zeros, None, loss, workspace=ws_q, d_status=dstat)
            mark("factor_and_quantize")
            g.gptq_pack(c, lin.bits, packed)
            mark("pack")
        return marks

    for _ in range(args.warmup):
        step(False)
    torch.cuda.synchronize()
    all_marks = []
    t0 = time.perf_counter()
    for _ in range(args.steps):
        all_marks.append(step(True))
    torch.cuda.synchronize()
    wall = time.perf_counter() - t0
    if int(dstat.item()) != 0:
        raise SystemExit(f"quantizer status {int(dstat.item())}: {g.gptq_status_string(int(dstat.item()))}")
    for marks in all_marks:
        for (_, a), (k, b) in zip(marks, marks[1:]):
            if k is not None:
                kinds[k].append(a.elapsed_time(b) / 1e3)
    step_s = wall / args.steps
    stage_s = {k: sum(v) / args.steps for k, v in kinds.items()}
    hess_flop = sum(a.tokens * a.n * (a.n + 1.0) for a in wl.hessians.values())
    fq_flop = 0.0
    current = None
    for lin in wl.linears:
        if lin.hessian != current:
            fq_flop += 2.0 * lin.cols ** 3 / 3.0
            current = lin.hessian
        fq_flop += float(lin.rows) * lin.cols * lin.cols
    hess_tflops = hess_flop / stage_s["hessian"] / 1e12
    x_bf16 = all(a.bf16 for a in wl.hessians.values())
    hess_peak = PEAK_BF16_TFLOPS if x_bf16 else PEAK_F32_TFLOPS
    nl = len(wl.linears)
    bits_mix = {str(b): sum(1 for l in wl.linears if l.bits == b) for b in sorted({l.bits for l in wl.linears})}
    tokens = sorted({a.tokens for a in wl.hessians.values()})
    return {
        "metric": METRIC,
        "value": nl / step_s,
        "unit": "layers/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": step_s * 1e3,
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16" if x_bf16 else "f32",
        "data": "synthetic",
        "config": {"workload": wl.description, "whole": True, "layers": nl, "hessians": len(wl.hessians),
                   "tokens": tokens[0] if len(tokens) == 1 else tokens, "bits": bits_mix,
                   "groupsize": wl.groupsize, "blocksize": wl.blocksize, "damp": wl.damp,
                   "inputs": "one generated tensor per shape; each Hessian and layer reads its own copy, "
                             "rolled by a distinct offset"},
        "stages_ms": {k: v * 1e3 for k, v in stage_s.items()},
        "stage_tflops": {"hessian_bf16_mfma" if x_bf16 else "hessian_f32_mfma": hess_tflops,
                         "factor_and_quantize_f32": fq_flop / stage_s["factor_and_quantize"] / 1e12},
        "roofline": {"bound": "mfma",
                     "kernel": ("k_syrk_bf16" if x_bf16 else "k_syrk_f32")
                               + " + k_syrk_reduce (every Hessian call of the pass)",
                     "achieved": hess_tflops, "peak": hess_peak, "unit": "TFLOP/s",
                     "frac": hess_tflops / hess_peak, "traffic": None},
        "input_generation_s": gen_s,
    }


def time_layer(args, g, torch, wl, lin, acts, bits, dev, workload_name, description=None):
    """Times args.steps passes over one layer (H = 0, Hessian, factor and quantize loop, pack)
    after args.warmup untimed ones, with the inputs resident in HBM.  Returns the record and the
    device tensors the measurements outside the step reuse."""
    rows, cols, tokens = lin.rows, lin.cols, acts.tokens
    t0 = time.perf_counter()
    X_bits = acts.full()
    W_bits = lin.weight()
    gen_s = time.perf_counter() - t0
    x_bf16 = acts.bf16
    Xd = host_tensor(torch, X_bits, x_bf16).to(dev)
    del X_bits
    Wd = host_tensor(torch, W_bits, lin.bf16).to(dev)
    params = g.Params(bits=bits, groupsize=wl.groupsize, blocksize=wl.blocksize, damp=wl.damp)
    G = -(-cols // wl.groupsize)
    H = torch.zeros((cols, cols), dtype=torch.float32, device=dev)
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, G), dtype=torch.float32, device=dev)
    zeros = torch.empty((rows, G), dtype=torch.uint8, device=dev)
    loss = torch.empty((rows,), dtype=torch.float32, device=dev)
    packed = torch.empty((rows, cols * bits // 32), dtype=torch.int32, device=dev)
    dstat = torch.zeros((1,), dtype=torch.int32, device=dev)
    ws_h = torch.empty(max(g.gptq_hessian_workspace_bytes(cols, tokens, g.GPTQ_BF16 if x_bf16 else g.GPTQ_F32), 1),
                       dtype=torch.uint8, device=dev)
    ws_q = torch.empty(g.gptq_quantize_workspace_bytes(rows, cols, params), dtype=torch.uint8, device=dev)

    if args.calib_copy:
        a = torch.empty(1 << 28, dtype=torch.float32, device=dev)  # 1 GiB
        b = torch.empty_like(a)
        b.copy_(a)
        torch.cuda.synchronize()
        del a, b

    ev = {k: [] for k in ("h0", "h1", "q1", "p1")}

    def step(record):
        H.zero_()
        if record:
            e = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
            e[0].record()
        g.gptq_accumulate_hessian(H, Xd, workspace=ws_h)
        if record:
            e[1].record()
        g.gptq_quantize_layer(Wd, H, params, codes, scales, zeros, None, loss, workspace=ws_q, d_status=dstat)
        if record:
            e[2].record()
        g.gptq_pack(codes, bits, packed)
        if record:
            e[3].record()
            for k, x in zip(("h0", "h1", "q1", "p1"), e):
                ev[k].append(x)

    for _ in range(args.warmup):
        step(False)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step(True)
    torch.cuda.synchronize()
    wall = time.perf_counter() - t0
    if int(dstat.item()) != 0:
        raise SystemExit(f"quantizer status {int(dstat.item())}: {g.gptq_status_string(int(dstat.item()))}")

    t_h = float(np.mean([a.elapsed_time(b) for a, b in zip(ev["h0"], ev["h1"])])) / 1e3
    t_q = float(np.mean([a.elapsed_time(b) for a, b in zip(ev["h1"], ev["q1"])])) / 1e3
    t_p = float(np.mean([a.elapsed_time(b) for a, b in zip(ev["q1"], ev["p1"])])) / 1e3
    step_s = wall / args.steps
    alg = algorithmic(rows, cols, tokens, bits)
    if not x_bf16:
        alg["x_bytes"] *= 2
    hess_peak = PEAK_BF16_TFLOPS if x_bf16 else PEAK_F32_TFLOPS
    hess_tflops = alg["hessian_flop"] / t_h / 1e12
    rec = {
        "metric": METRIC,
        "value": 1.0 / step_s,
        "unit": "layers/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": step_s * 1e3,
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "bf16" if x_bf16 else "f32",
        "data": "synthetic",
        "config": {"workload": description or wl.description, "layer": lin.name, "rows": rows, "cols": cols,
                   "tokens": tokens, "bits": bits, "groupsize": wl.groupsize, "blocksize": wl.blocksize,
                   "damp": wl.damp},
        "tflops": alg["total_flop"] / step_s / 1e12,
        "stages_ms": {"hessian": t_h * 1e3, "factor_and_quantize": t_q * 1e3, "pack": t_p * 1e3},
        "stage_tflops": {"hessian_bf16_mfma" if x_bf16 else "hessian_f32_mfma": hess_tflops,
                         "factor_and_quantize_f32": (alg["factor_flop"] + alg["quantize_flop"]) / t_q / 1e12},
        "quantize_only_layers_per_s": 1.0 / (t_q + t_p),
        "roofline": {"bound": "mfma",
                     "kernel": ("k_syrk_bf16" if x_bf16 else "k_syrk_f32") + " + k_syrk_reduce (one Hessian call)",
                     "achieved": hess_tflops,
                     "peak": hess_peak, "unit": "TFLOP/s", "frac": hess_tflops / hess_peak,
                     "traffic": syrk_traffic(workload_name, tokens),
                     "algorithmic_bytes": alg["x_bytes"] + 8.0 * cols * cols},  # X read, H read and written
        "input_generation_s": gen_s,
    }
    state = {"W_bits": W_bits, "Xd": Xd, "Wd": Wd, "packed": packed, "scales": scales, "zeros": zeros,
             "x_bf16": x_bf16, "w_bf16": lin.bf16}
    return rec, state


TRACE_REC = 32  # words per trace record (gptq_trace_set in include/gptq.h)
TRACE_LOOP, TRACE_POTRF, TRACE_TRSM, TRACE_DIAG, TRACE_TILE, TRACE_MMA = 1, 2, 3, 4, 5, 6


def trace_summary(words, count):
    """Decodes the trace buffer (uint64 words as gptq_trace_set lays them out) into phase medians
    in microseconds (the stamps are a 100 MHz clock).  Host logic only."""
    words = np.asarray(words, dtype=np.int64)
    n = min(int(count), int(words[0]))
    rec = words[TRACE_REC:TRACE_REC * (n + 1)].reshape(n, TRACE_REC)
    kind, tag, cnt, st = rec[:, 0], rec[:, 2], rec[:, 3], rec[:, 4:].astype(np.float64) / 100.0
    med = lambda v: float(np.median(v)) if len(v) else None  # noqa: E731
    out = {"records": int(count), "kept": n}
    lp = st[(kind == TRACE_LOOP) & (cnt >= 7) & (tag >= 1)]
    names = ("operands_and_near_update", "stores_to_lds", "barrier", "update_applied_and_group_range",
             "steps_128", "outputs")
    out["loop_workgroup_us"] = {nm: med(lp[:, i + 1] - lp[:, i]) for i, nm in enumerate(names)}
    out["loop_workgroup_us"]["total"] = med(lp[:, 6] - lp[:, 0])
    po = st[(kind == TRACE_POTRF) & (cnt >= 18)]
    ptag = tag[(kind == TRACE_POTRF) & (cnt >= 18)]
    if len(po):
        panels = sum(po[:, 2 + 2 * p] - (po[:, 1] if p == 0 else po[:, 1 + 2 * p]) for p in range(8))
        updates = sum(po[:, 3 + 2 * p] - po[:, 2 + 2 * p] for p in range(7))
        late = ptag >= 10
        out["diagonal_factor_us"] = {"load": med(po[:, 1] - po[:, 0]), "panels": med(panels),
                                     "updates": med(updates), "write": med(po[:, 17] - po[:, 16]),
                                     "total": med(po[:, 17] - po[:, 0]),
                                     "total_late_steps": med((po[:, 17] - po[:, 0])[late])}
    tr = kind == TRACE_TRSM
    if tr.any():
        out["block_solve_workgroup_us"] = {"fill_and_rows": med(st[tr, 1] - st[tr, 0]),
                                           "steps_128": med(st[tr, 2] - st[tr, 1])}
    # the chain, step by step: diagonal factor k -> solve k -> update of block k+1 -> factor k+1
    spans = {}
    for kd in (TRACE_POTRF, TRACE_TRSM, TRACE_DIAG, TRACE_TILE):
        sel = kind == kd
        last = np.where(cnt[sel] > 0, st[sel, np.maximum(cnt[sel] - 1, 0)], 0.0)
        for t, a, b in zip(tag[sel], st[sel, 0], last):
            lo, hi = spans.get((kd, int(t)), (np.inf, -np.inf))
            spans[(kd, int(t))] = (min(lo, a), max(hi, b))
    gaps, solve, diag, tiles = [], [], [], []
    for k in sorted(t for (kd, t) in spans if kd == TRACE_POTRF):
        if (TRACE_TRSM, k) not in spans or (TRACE_DIAG, k + 1) not in spans or (TRACE_POTRF, k + 1) not in spans:
            continue
        p0, p1 = spans[(TRACE_POTRF, k)]
        s0, s1 = spans[(TRACE_TRSM, k)]
        d0, d1 = spans[(TRACE_DIAG, k + 1)]
        n0 = spans[(TRACE_POTRF, k + 1)][0]
        gaps.append((s0 - p1) + (d0 - s1) + (n0 - d1))
        solve.append(s1 - s0)
        diag.append(d1 - d0)
        if (TRACE_TILE, k + 1) in spans:
            tiles.append(spans[(TRACE_TILE, k + 1)][1] - spans[(TRACE_TILE, k + 1)][0])
    out["chain_step_us"] = {"solve_span": med(solve), "diagonal_update_span": med(diag),
                            "gaps_between_launches": med(gaps), "step_tiles_span": med(tiles), "steps": len(gaps)}
    return out


def trace_batch_summary(words, count):
    """Decodes the matrix-core batch product's records (kind 6: one a workgroup, stamps at its start,
    after its x loads, after its scale and code loads, after the LDS zeroing, after staging, after the
    chunks, at its end) into phase medians and percentiles in microseconds, the workgroups' start and
    life times relative to the first start, and how many were alive at 12 points of the kernel's span.
    Host logic only."""
    words = np.asarray(words, dtype=np.int64)
    n = min(int(count), int(words[0]))
    rec = words[TRACE_REC:TRACE_REC * (n + 1)].reshape(n, TRACE_REC)
    rec = rec[(rec[:, 0] == TRACE_MMA) & (rec[:, 3] >= 7)]
    if not len(rec):
        return {"workgroups": 0}
    st = rec[:, 4:11].astype(np.float64) / 100.0
    st -= st[:, 0].min()
    ph = np.diff(st, axis=1)
    names = ("x_loads_issued", "scale_and_code_loads_issued", "lds_zeroed", "staged", "chunks_applied",
             "rows_combined_and_written")
    span = float(st[:, 6].max())
    pct = lambda v: [float(np.percentile(v, q)) for q in (0, 25, 50, 75, 100)]  # noqa: E731
    return {"workgroups": int(len(rec)), "kernel_span_us": span,
            "start_us_percentiles": pct(st[:, 0]), "lifetime_us_percentiles": pct(st[:, 6] - st[:, 0]),
            "phase_median_us": {nm: float(np.median(ph[:, i])) for i, nm in enumerate(names)},
            "phase_p90_us": {nm: float(np.percentile(ph[:, i], 90)) for i, nm in enumerate(names)},
            "alive": [int(((st[:, 0] <= t) & (st[:, 6] > t)).sum()) for t in np.linspace(0.0, span, 12)]}


def trace_batch(g, torch, dev, rows=5120, cols=25600, batch=8, bits=4, groupsize=128):
    """One call of the batch product (5120x25600, 4-bit g128, 8 fp32 vectors, seeded random codes,
    scales and zeros) on the trace build, after one untimed call."""
    gen = torch.Generator(dev).manual_seed(5)
    G = -(-cols // groupsize)
    packed = torch.randint(-2 ** 31, 2 ** 31 - 1, (rows, cols * bits // 32), dtype=torch.int32, device=dev,
                           generator=gen)
    scales = 0.005 + 0.015 * torch.rand((rows, G), device=dev, generator=gen)
    zeros = torch.randint(0, 2 ** bits, (rows, G), dtype=torch.uint8, device=dev, generator=gen)
    X = torch.randn(batch, cols, device=dev, generator=gen)
    Y = torch.empty(batch, rows, device=dev)
    g.gptq_dequant_gemm(packed, scales, zeros, bits, groupsize, X, Y)
    cap = 1 << 14
    buf = torch.zeros(TRACE_REC * (cap + 1), dtype=torch.int64, device=dev)
    buf[0] = cap
    torch.cuda.synchronize()
    g.gptq_trace_set(buf)
    g.gptq_dequant_gemm(packed, scales, zeros, bits, groupsize, X, Y)
    torch.cuda.synchronize()
    g.gptq_trace_set(None)
    words = buf.cpu().numpy()
    out = trace_batch_summary(words, int(words[1]))
    out["config"] = {"rows": rows, "cols": cols, "batch": batch, "bits": bits, "groupsize": groupsize,
                     "x": "fp32"}
    return out


def trace_layer(args, g, torch, wl, lin, acts, bits, dev):
    """One pass of the layer (Hessian, factor, quantize) on the trace build, after one untimed pass."""
    Xd = host_tensor(torch, acts.full(), acts.bf16).to(dev)
    Wd = host_tensor(torch, lin.weight(), lin.bf16).to(dev)
    params = g.Params(bits=bits, groupsize=wl.groupsize, blocksize=wl.blocksize, damp=wl.damp)
    H = torch.zeros((lin.cols, lin.cols), dtype=torch.float32, device=dev)
    g.gptq_accumulate_hessian(H, Xd)
    g.quantize(Wd, H, params)
    cap = 1 << 18
    buf = torch.zeros(TRACE_REC * (cap + 1), dtype=torch.int64, device=dev)
    buf[0] = cap
    torch.cuda.synchronize()
    g.gptq_trace_set(buf)
    H.zero_()
    g.gptq_accumulate_hessian(H, Xd)
    g.quantize(Wd, H, params)
    torch.cuda.synchronize()
    g.gptq_trace_set(None)
    words = buf.cpu().numpy()
    out = trace_summary(words, int(words[1]))
    out["config"] = {"workload": wl.description, "layer": lin.name, "rows": lin.rows, "cols": lin.cols, "bits": bits}
    return out


def main():
    args = parse()
    if args.gpus != 1:
        print(f"bench.py: this build runs on one GPU; --gpus {args.gpus} is not supported "
              "(the Hessian would shard by tokens with one reduction, rows and layers are independent; "
              "see the design notes)", file=sys.stderr)
        sys.exit(2)

    import torch

    import post_weight_quantization_03_amd as g
    from post_weight_quantization_03_amd import synth

    wl = synth.workload(args.workload, tokens=args.tokens)
    dev = torch.device("cuda:0")
    if args.trace:
        g.LIB_PATH = os.path.join(os.path.dirname(g.__file__), "libgptq_trace.so")
        lin = wl.linears[args.layer]
        print(json.dumps({"trace": trace_layer(args, g, torch, wl, lin, wl.hessians[lin.hessian], lin.bits, dev),
                          "batch_product": trace_batch(g, torch, dev)}), flush=True)
        return
    if args.whole:
        print(json.dumps(whole_workload(args, g, torch, wl, dev)), flush=True)
        return
    lin = wl.linears[args.layer]
    acts = wl.hessians[lin.hessian]
    rows, cols, tokens, bits = lin.rows, lin.cols, acts.tokens, lin.bits
    rec, st = time_layer(args, g, torch, wl, lin, acts, bits, dev, args.workload)
    if not args.no_extras and not (st["x_bf16"] and st["w_bf16"]):
        rec["extras"] = "skipped: the rotation, correction and GEMV measurements take bf16 weights and activations"
    elif not args.no_extras:
        # measurements outside the timed step; a failure is reported in its field and
        # does not take the step's line with it
        extras = {
            "hadamard_rotation": lambda: hadamard_measure(g, torch, st["Wd"], cols, dev),
            "qep_correction": lambda: qep_measure(g, torch, st["Xd"], st["Wd"], cols, dev),
            "dequant_gemv": lambda: gemv_measure(g, torch, st["packed"], st["scales"], st["zeros"], rows, cols,
                                                 bits, wl.groupsize, dev),
            "dequant_gemv_shapes": lambda: gemv_shapes_measure(g, torch, dev),
        }
        for name, fn in extras.items():
            try:
                rec[name] = fn()
            except Exception as ex:  # noqa: BLE001
                rec[name] = {"error": f"{type(ex).__name__}: {ex}"}
                print(f"bench.py: {name} failed: {ex}", file=sys.stderr)
            torch.cuda.empty_cache()
    W_bits = st["W_bits"]
    x_bf16, w_bf16 = st["x_bf16"], st["w_bf16"]
    del st
    torch.cuda.empty_cache()
    if args.workload == "q_proj_4096" and args.layer == 0 and args.tokens is None and not args.no_second:
        # the metric's second shape: a Llama-2-7B gate_proj-shaped layer (11008 x 4096) at 4-bit
        # g128, on its own 131072-token Hessian of the MLP input law
        wl2 = synth.workload("mlp_7b")
        lin2 = wl2.linears[0]
        desc = ("Llama-2-7B gate_proj 11008x4096 bf16 ~N(0,0.02^2), X 131072x4096 bf16 t4 with 41 outlier "
                "channels x20, 4-bit g128")
        rec2, st2 = time_layer(args, g, torch, wl2, lin2, wl2.hessians[lin2.hessian], 4, dev, "gate_proj_4bit",
                               desc)
        del st2
        torch.cuda.empty_cache()
        rec["shape_11008x4096"] = {k: rec2[k] for k in ("value", "unit", "ms_per_step", "config", "tflops",
                                                        "stages_ms", "stage_tflops", "quantize_only_layers_per_s",
                                                        "roofline")}
        rec["both_shapes_layers_per_s"] = 2.0 / (rec["ms_per_step"] / 1e3 + rec2["ms_per_step"] / 1e3)
    if not args.no_cpu_baseline:
        rec["cpu_baseline"] = cpu_baseline(W_bits, acts, rows, cols, tokens, bits, args, x_bf16, w_bf16)
    print(json.dumps(rec), flush=True)


if __name__ == "__main__":
    main()
