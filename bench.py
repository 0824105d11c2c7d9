#!/usr/bin/env python3
"""Benchmark of the attention hot path on GB300.

One step = one forward + one backward (atomic-dQ mode) of exact causal
attention on the bf16 training shape b=4, s=8192, hq=32, hkv=8, d=128
(GQA 4:1), inputs resident in HBM.  The headline value is TFLOP/s counted
with the FlashAttention FAQ's causal formula (Inference Cookbook Q16):
4*b*hq*s*s*d/2 for the forward and 2.5x that for the backward.

Also measured on the same run (each in its own timed loop): forward alone,
backward alone, the deterministic backward, the varlen workload, the paged
decode workload (HBM GB/s), an end-to-end pass through the public API from
pinned host buffers, and the float64 CPU oracle on a bounded sample.

Usage: python bench.py [--gpus N] [--steps K] [--warmup W] [--impl reference]
       python bench.py --profile-case fwd|bwd|decode|varlen|paged|norm|norm_bwd
           (one small case for ncu)
Under torchrun each rank runs its own replica (weak scaling) and rank 0
prints one JSON line.
"""
from __future__ import annotations

import argparse
import hashlib
import json
import math
import os
import statistics
import subprocess
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

METRIC = "attention fwd/fwd+bwd TFLOP/s, bf16 causal N=8k d=128; % of GB300 tensor peak"
B, S, HQ, HKV, D = 4, 8192, 32, 8, 128
FWD_FLOPS = 4 * B * HQ * S * S * D / 2          # 2.199e12
BWD_FLOPS = 2.5 * FWD_FLOPS                     # 5.498e12
STEP_FLOPS = FWD_FLOPS + BWD_FLOPS
WORKLOAD = "training fwd+bwd, bf16, causal, b=4 s=8192 hq=32 hkv=8 d=128 (GQA 4:1), atomic dQ"


def peaks():
    try:
        with open(os.path.join(ROOT, "MEASURED_PEAKS.json")) as f:
            p = json.load(f)
        return {"hbm_gbs": p["hbm_gbs"], "bf16_tflops": p["bf16_tflops"],
                "bf16_tflops_sustained": p.get("bf16_tflops_sustained", p["bf16_tflops"]),
                "source": "measured"}
    except (OSError, KeyError, ValueError):
        return {"hbm_gbs": 6800.0, "bf16_tflops": 1900.0, "bf16_tflops_sustained": 1700.0,
                "source": "fallback"}


# ------------------------------------------------------------------ clocks


class ClockSampler:
    """nvidia-smi samples (200 ms) while a timed region runs."""

    FIELDS = ("clocks.sm,clocks.max.sm,power.draw,clocks_event_reasons.hw_slowdown,"
              "clocks_event_reasons.hw_thermal_slowdown,clocks_event_reasons.sw_thermal_slowdown,"
              "clocks_event_reasons.sw_power_cap")

    def __init__(self, index: int):
        self.index = index
        self.proc = None

    def __enter__(self):
        try:
            self.proc = subprocess.Popen(
                ["nvidia-smi", f"--query-gpu={self.FIELDS}", "--format=csv,noheader,nounits",
                 "-lms", "200", "-i", str(self.index)],
                stdout=subprocess.PIPE, stderr=subprocess.DEVNULL, text=True)
        except OSError:
            self.proc = None
        time.sleep(0.3)
        return self

    def __exit__(self, *exc):
        self.lines = []
        if self.proc is not None:
            time.sleep(0.25)
            self.proc.terminate()
            try:
                out, _ = self.proc.communicate(timeout=5)
            except subprocess.TimeoutExpired:
                self.proc.kill()
                out, _ = self.proc.communicate()
            self.lines = [l for l in out.splitlines() if l.strip()]
        return False

    def summary(self):
        sm, mx, reasons = [], None, set()
        names = ["hw_slowdown", "hw_thermal_slowdown", "sw_thermal_slowdown", "sw_power_cap"]
        for line in self.lines:
            parts = [p.strip() for p in line.split(",")]
            if len(parts) < 7:
                continue
            try:
                sm.append(float(parts[0]))
                mx = float(parts[1])
            except ValueError:
                continue
            for n, v in zip(names, parts[3:7]):
                if v.lower().startswith("active"):
                    reasons.add(n)
        return {"sm_mhz": statistics.median(sm) if sm else None, "sm_max_mhz": mx,
                "reasons": sorted(reasons), "samples": len(sm)}


# ------------------------------------------------------------------ helpers


def sources_sha(names):
    h = hashlib.sha256()
    for n in names:
        with open(os.path.join(ROOT, "exact_attention_41_gb300", "csrc", n), "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


TRAFFIC_NOTE = ("DRAM bytes seen during one launch (dram__bytes_read + dram__bytes_write, "
                "ncu capture of the b=1 case scaled by 4); writes still held in L2 when the "
                "kernel ends are not in it")


def traffic_for(kernel_key):
    """DRAM bytes per launch from a committed ncu summary, if the kernel's
    sources are unchanged since that capture; else None."""
    try:
        with open(os.path.join(ROOT, "profiles", "dram_traffic.json")) as f:
            t = json.load(f)[kernel_key]
        if sources_sha(t["sources"]) != t["sources_sha256"]:
            return None
        return t["bytes_per_launch"]
    except (OSError, KeyError, ValueError):
        return None


def max_over_ranks(ms, world, device=None):
    """The job's step time: the slowest rank's (a MAX all-reduce); with one
    rank, the local time."""
    if world <= 1:
        return ms
    import torch
    import torch.distributed as dist

    t = torch.tensor([ms], dtype=torch.float64, device=device)
    dist.all_reduce(t, op=dist.ReduceOp.MAX)
    return float(t.item())


def job_value(step_flops, ms, world):
    """Whole-job TFLOP/s: every rank runs its own replica of the step."""
    return world * step_flops / (ms * 1e-3) / 1e12


def timed(fn, steps, stream):
    import torch

    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record(stream)
    for _ in range(steps):
        fn()
    end.record(stream)
    torch.cuda.synchronize()
    return start.elapsed_time(end) / steps


def dev_normal(shape, seed, dtype):
    import torch

    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


# ------------------------------------------------------------------ workloads


def training_inputs():
    import torch

    bf = torch.bfloat16
    q = dev_normal((B, S, HQ, D), 60, bf)
    k = dev_normal((B, S, HKV, D), 61, bf)
    v = dev_normal((B, S, HKV, D), 62, bf)
    do = dev_normal((B, S, HQ, D), 63, bf)
    return q, k, v, do


def bench_varlen(libattn, steps, stream):
    import numpy as np
    import torch

    from exact_attention_41_gb300 import synthetic as syn

    lens = syn.varlen_lengths(7)
    cu = torch.from_numpy(syn.cu_seqlens(lens)).cuda()
    t = int(lens.sum())
    bf = torch.bfloat16
    q, k, v, do = (dev_normal((t, h, D), 70 + i, bf) for i, h in enumerate((HQ, HKV, HKV, HQ)))
    kw = dict(causal=True, window=(256, 0), softcap=50.0)
    mx = int(lens.max())
    o, lse = libattn.fwd_varlen(q, k, v, cu, cu, mx, mx, **kw)
    ws = torch.empty(libattn.lib().attn_bwd_varlen_workspace_size(len(lens), mx, mx, t, t, HQ,
                                                                  HKV, D, 0),
                     device="cuda", dtype=torch.uint8)
    # visible (query, key) pairs per head: sum over sequences of min(i + 1, 257)
    pairs = sum(int(np.minimum(np.arange(n) + 1, 257).sum()) for n in lens)
    flops_f = 4.0 * HQ * D * pairs

    def f():
        libattn.fwd_varlen(q, k, v, cu, cu, mx, mx, out=o, lse=lse, **kw)

    def fb():
        f()
        libattn.bwd_varlen(q, k, v, o, lse, do, cu, cu, mx, mx, workspace=ws, **kw)

    for _ in range(2):
        fb()
    tf = timed(f, steps, stream)
    tfb = timed(fb, steps, stream)
    return {"workload": "varlen 64 seqs U[100,4096] (seed 7), bf16, hq=32 hkv=8 d=128, causal, "
                        "window (256,0), softcap 50",
            "tokens": t, "visible_pairs_per_head": pairs,
            "fwd_ms": round(tf, 4), "fwd_tflops": round(flops_f / tf / 1e9, 2),
            "fwd_bwd_ms": round(tfb, 4), "fwd_bwd_tflops": round(3.5 * flops_f / tfb / 1e9, 2),
            "flops_note": "algorithmic: 4*hq*d*visible pairs (fwd), x2.5 bwd"}


def bench_head_dims(libattn, steps, stream):
    """Forward and backward TFLOP/s at head dims 64 and 256 beside 128, on a
    causal bf16 problem of the training shape's kind (b=2, s=4096, GQA 4:1,
    hq * d = 4096), both dQ modes, all on the tensor cores."""
    import torch

    out = {}
    b, s = 2, 4096
    for d, hq in ((64, 64), (128, 32), (256, 16)):
        hkv = hq // 4
        q, do = (dev_normal((b, s, hq, d), 90 + i, torch.bfloat16) for i in range(2))
        k, v = (dev_normal((b, s, hkv, d), 92 + i, torch.bfloat16) for i in range(2))
        o, lse = libattn.fwd(q, k, v, causal=True)
        ws = libattn.bwd_workspace(q, k, False)
        ws_det = libattn.bwd_workspace(q, k, True)
        grads = [torch.empty_like(x) for x in (q, k, v)]
        flops = 4.0 * b * hq * s * s * d / 2

        def f():
            libattn.fwd(q, k, v, causal=True, out=o, lse=lse)

        def g(det=False):
            libattn.bwd(q, k, v, o, lse, do, causal=True, deterministic=det,
                        workspace=ws_det if det else ws, dq=grads[0], dk=grads[1], dv=grads[2])

        f()
        g()
        g(True)
        tf, tb = timed(f, steps, stream), timed(g, steps, stream)
        td = timed(lambda: g(True), steps, stream)
        out[f"d{d}"] = {"fwd_ms": round(tf, 4), "fwd_tflops": round(flops / tf / 1e9, 2),
                        "bwd_ms": round(tb, 4), "bwd_tflops": round(2.5 * flops / tb / 1e9, 2),
                        "bwd_deterministic_ms": round(td, 4),
                        "bwd_deterministic_tflops": round(2.5 * flops / td / 1e9, 2)}
        del q, do, k, v, o, lse, ws, ws_det, grads
        torch.cuda.empty_cache()
    out["workload"] = ("causal bf16 b=2 s=4096, (hq, d) in {(64, 64), (32, 128), (16, 256)}, "
                       "hkv = hq / 4")
    return out


def bench_decode(libattn, steps, stream, sq):
    import numpy as np
    import torch

    from exact_attention_41_gb300 import synthetic as syn

    b, page = 64, 256
    seqlens, table, npages = syn.decode_layout(8, b, 32768, page, sq)
    bf = torch.bfloat16
    kc = dev_normal((npages, page, HKV, D), 80, bf)
    vc = dev_normal((npages, page, HKV, D), 81, bf)
    q = dev_normal((b, sq, HQ, D), 82, bf)
    kn = dev_normal((b, sq, HKV, D), 83, bf)
    vn = dev_normal((b, sq, HKV, D), 84, bf)
    sl = torch.from_numpy(seqlens).cuda()
    bt = torch.from_numpy(table).cuda()
    splits = libattn.num_splits(b, sq, HQ, HKV, D, table.shape[1] * page, 0)
    ws = libattn.kvcache_workspace(q, kc, page, table.shape[1], 0)
    o = torch.empty_like(q)
    lse = torch.empty((b, HQ, sq), device="cuda", dtype=torch.float32)

    def f():
        libattn.fwd_kvcache(q, kc, vc, sl, k_new=kn, v_new=vn, block_table=bt, causal=True,
                            workspace=ws, out=o, lse=lse)

    for _ in range(3):
        f()
    # flush L2 between reps is unnecessary: 8.6 GB of K/V per step >> L2
    t = timed(f, steps, stream)
    kv_bytes = int((seqlens.astype(np.int64) + sq).sum()) * HKV * D * 2 * 2
    io_bytes = (2 * b * sq * HQ * D * 2 + b * HQ * sq * 4      # q read, out write, lse
                + 2 * b * sq * HKV * D * 2)                    # k_new/v_new read (cache write
    #                                                            counted in kv_bytes read side)
    total = kv_bytes + io_bytes
    return {"workload": f"paged decode bf16 b=64 sq=s_new={sq} hq=32 hkv=8 d=128, "
                        "cache_seqlens U[1,32768] (seed 8), 256-token pages, causal",
            "num_splits": splits, "ms": round(t, 4), "bytes": total,
            "gbs": round(total / t / 1e6, 1), "tokens_per_s": round(b * sq / t * 1e3, 1)}


def cpu_baseline_sample(repeat=1):
    """The float64 oracle on a bounded sample of the training workload: the
    forward and backward of one (batch, head) at s=8192, causal."""
    import numpy as np

    from exact_attention_41_gb300 import synthetic as syn
    from oracle import attention as ref

    rng = np.random.default_rng(90)
    q, k, v, do = (syn.bits_to_f64(syn.normal_bits(rng, (S, D), syn.BF16), syn.BF16)
                   for _ in range(4))
    t0 = time.perf_counter()
    for _ in range(repeat):
        ref.head_forward(q, k, v, np.arange(S), S, S, 1 / math.sqrt(D), causal=True)
        ref.head_backward(q, k, v, do, S, S, 1 / math.sqrt(D), causal=True)
    dt = (time.perf_counter() - t0) / repeat
    flops = STEP_FLOPS / (B * HQ)
    n1 = 4096
    t1 = one_thread_seconds(n1)
    flops1 = 3.5 * 4 * n1 * n1 * D / 2
    return {"value": round(flops / dt / 1e12, 6), "unit": "TFLOP/s", "cores": os.cpu_count(),
            "kind": "oracle",
            "sample": "float64 oracle fwd+bwd of one (batch, head) of the training shape "
                      f"(s=8192, d=128, causal), {dt:.2f} s; algorithmic causal FLOPs "
                      f"{flops:.3e}; numpy/BLAS on all host threads",
            "one_thread": None if t1 is None else {
                "value": round(flops1 / t1 / 1e12, 6), "unit": "TFLOP/s", "seconds": round(t1, 2),
                "sample": f"the same on the causal prefix of {n1} tokens, one BLAS thread"},
            "cpu": cpu_info()}


def bench_e2e(libattn, inputs, fwd_bwd_into, steps, stream):
    """The training step through the public API with the data on the host:
    every step uploads its q, k, v, dO from pinned host memory and reads its
    dq, dk, dv back into pinned host memory.  Device buffers are doubled so
    that the uploads of step i+1 and the downloads of step i-1 run on two copy
    streams while step i computes; the first upload and the last download are
    inside the timed region too.  Afterwards the downloaded gradients are
    compared with an eager step on the same inputs."""
    import torch

    host_in = [x.cpu().pin_memory() for x in inputs]
    bufs = [[torch.empty_like(x) for x in inputs] for _ in range(2)]
    grads = [[torch.empty_like(x) for x in inputs[:3]] for _ in range(2)]
    host_out = [torch.empty(x.shape, dtype=x.dtype).pin_memory() for x in inputs[:3]]
    h2d = sum(x.numel() * x.element_size() for x in host_in)
    d2h = sum(x.numel() * x.element_size() for x in host_out)
    up, down = torch.cuda.Stream(), torch.cuda.Stream()
    ev = lambda: torch.cuda.Event()
    up_done, comp_done, down_done = [ev(), ev()], [ev(), ev()], [ev(), ev()]

    def run(n):
        main = torch.cuda.current_stream()
        up.wait_stream(main)
        down.wait_stream(main)
        for i in range(n):
            s = i % 2
            with torch.cuda.stream(up):
                if i >= 2:
                    up.wait_event(comp_done[s])  # step i-2 no longer reads set s
                for d, h in zip(bufs[s], host_in):
                    d.copy_(h, non_blocking=True)
                up_done[s].record(up)
            main.wait_event(up_done[s])
            if i >= 2:
                main.wait_event(down_done[s])    # step i-2's gradients are read out
            fwd_bwd_into(*bufs[s], *grads[s])
            comp_done[s].record(main)
            with torch.cuda.stream(down):
                down.wait_event(comp_done[s])
                for h, d in zip(host_out, grads[s]):
                    h.copy_(d, non_blocking=True)
                down_done[s].record(down)
        main.wait_stream(up)
        main.wait_stream(down)

    run(2)
    ms = timed(lambda: run(steps), 1, stream) / steps
    torch.cuda.synchronize()
    # the last step's downloaded gradients against an eager step
    ref = [torch.empty_like(x) for x in inputs[:3]]
    fwd_bwd_into(*inputs, *ref)
    torch.cuda.synchronize()
    same_kv = all(torch.equal(h.cuda().view(torch.int16), r.view(torch.int16))
                  for h, r in zip(host_out[1:], ref[1:]))
    dq_ok = torch.allclose(host_out[0].cuda().float(), ref[0].float(), atol=1e-2, rtol=1e-2)
    info = {"h2d_bytes_per_step": h2d, "d2h_bytes_per_step": d2h,
            "overlap": "double-buffered device inputs/gradients; uploads and downloads on two "
                       "copy streams overlap the neighbouring steps' compute",
            "check": {"dk_dv_bitwise_equal_to_eager": bool(same_kv),
                      "dq_within_1e-2_of_eager": bool(dq_ok)}}
    del host_in, bufs, grads, host_out
    return ms, info


def accuracy_sample(libattn, inputs, o, lse, ws):
    """Error of the training step against the float64 oracle on one (batch,
    KV head) group -- the forward output and the gradients, against the
    oracle's stored-O reading of D and against the exact gradient -- as the
    worst error/bound ratio and the fraction out of bound for the contract
    (bf16: 1e-2 + 1e-2 |ref|) and for the Inference Cookbook FAQ Q10 bf16
    tolerance (5e-3 + 5e-3 |ref|).  Reported, not asserted."""
    import numpy as np
    import torch

    from oracle import attention as ref

    q, k, v, do = inputs
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    libattn.fwd(q, k, v, causal=True, out=o, lse=lse)
    libattn.bwd(q, k, v, o, lse, do, causal=True, workspace=ws, dq=dq, dk=dk, dv=dv)
    torch.cuda.synchronize()
    bi, kv, g = 1, 3, HQ // HKV
    hs = slice(kv * g, (kv + 1) * g)
    t0 = time.perf_counter()
    f64 = lambda t: t.double().cpu().numpy()
    qg, dog = f64(q[bi:bi + 1, :, hs]), f64(do[bi:bi + 1, :, hs])
    kg, vg = f64(k[bi:bi + 1, :, kv:kv + 1]), f64(v[bi:bi + 1, :, kv:kv + 1])
    scale = 1 / math.sqrt(D)
    ro, _ = ref.forward(qg, kg, vg, scale, causal=True)
    stored = ref.backward(qg, kg, vg, dog, scale, causal=True, stored_o="bf16")
    exact = ref.backward(qg, kg, vg, dog, scale, causal=True)
    got = {"O": f64(o[bi:bi + 1, :, hs]), "dQ": f64(dq[bi:bi + 1, :, hs]),
           "dK": f64(dk[bi:bi + 1, :, kv:kv + 1]), "dV": f64(dv[bi:bi + 1, :, kv:kv + 1])}

    def stats(x, r):
        err = np.abs(x - r)
        res = {"max_abs_err": float(err.max())}
        for name, tol in (("contract", 1e-2), ("pages_q10", 5e-3)):
            bound = tol + tol * np.abs(r)
            res[name] = {"worst_ratio": round(float((err / bound).max()), 4),
                         "frac_out": float((err > bound).mean())}
        return res

    res = {"sample": f"batch {bi}, kv head {kv} (query heads {hs.start}-{hs.stop - 1}) of the "
                     "training step, all 8192 rows, atomic dQ",
           "O": stats(got["O"], ro)}
    for n, i in (("dQ", 0), ("dK", 1), ("dV", 2)):
        res[n + "_vs_stored_o"] = stats(got[n], stored[i])
        res[n + "_vs_exact"] = stats(got[n], exact[i])
    res["oracle_seconds"] = round(time.perf_counter() - t0, 1)
    return res


def cpu_info():
    """Host CPU model, architecture and thread count (for the baseline)."""
    import platform

    model = None
    try:
        out = subprocess.run(["lscpu"], capture_output=True, text=True, timeout=10).stdout
        for line in out.splitlines():
            if line.startswith("Model name:"):
                model = line.split(":", 1)[1].strip()
                break
    except (OSError, subprocess.SubprocessError):
        pass
    return {"model": model, "arch": platform.machine(), "nproc": os.cpu_count()}


ONE_THREAD_SNIPPET = """
import math, sys, time
import numpy as np
sys.path.insert(0, {root!r})
from exact_attention_41_gb300 import synthetic as syn
from oracle import attention as ref
n, d = {n}, {d}
rng = np.random.default_rng(90)
q, k, v, do = (syn.bits_to_f64(syn.normal_bits(rng, (n, d), syn.BF16), syn.BF16) for _ in range(4))
t0 = time.perf_counter()
ref.head_forward(q, k, v, np.arange(n), n, n, 1 / math.sqrt(d), causal=True)
ref.head_backward(q, k, v, do, n, n, 1 / math.sqrt(d), causal=True)
print(time.perf_counter() - t0)
"""


def one_thread_seconds(n):
    """The oracle's fwd+bwd of one (batch, head) causal prefix of n tokens in
    a child process limited to one BLAS/OpenMP thread; None if it fails."""
    env = dict(os.environ, OMP_NUM_THREADS="1", OPENBLAS_NUM_THREADS="1", MKL_NUM_THREADS="1")
    try:
        r = subprocess.run([sys.executable, "-c", ONE_THREAD_SNIPPET.format(root=ROOT, n=n, d=D)],
                           capture_output=True, text=True, env=env, timeout=300)
        return float(r.stdout.strip().splitlines()[-1])
    except (OSError, subprocess.SubprocessError, ValueError, IndexError):
        return None


# ------------------------------------------------------------------ arms


def run_reference(args, rank):
    """The float64 oracle as it stands, on the host cores: each step is a
    bounded sample of the training workload, the causal attention (forward
    and backward) of the first 4096 tokens of one (batch, head)."""
    if rank != 0:
        return
    import numpy as np

    from exact_attention_41_gb300 import synthetic as syn
    from oracle import attention as ref

    n = 4096
    rng = np.random.default_rng(90)
    q, k, v, do = (syn.bits_to_f64(syn.normal_bits(rng, (n, D), syn.BF16), syn.BF16)
                   for _ in range(4))

    def step():
        ref.head_forward(q, k, v, np.arange(n), n, n, 1 / math.sqrt(D), causal=True)
        ref.head_backward(q, k, v, do, n, n, 1 / math.sqrt(D), causal=True)

    for _ in range(args.warmup):
        step()
    t0 = time.perf_counter()
    for _ in range(args.steps):
        step()
    dt = (time.perf_counter() - t0) / args.steps
    flops = 3.5 * 4 * n * n * D / 2
    value = flops / dt / 1e12
    sample = (f"float64 oracle fwd+bwd per step of the causal prefix of {n} tokens of one "
              "(batch, head) of the training shape (d=128); algorithmic causal FLOPs "
              f"{flops:.3e}; numpy/BLAS on all host threads")
    print(json.dumps({
        "impl": "reference", "metric": METRIC, "value": round(value, 6), "unit": "TFLOP/s",
        "n_gpus": args.gpus, "steps": args.steps, "warmup": args.warmup,
        "ms_per_step": round(dt * 1e3, 2), "higher_is_better": True, "scaling": "weak",
        "vs_baseline": None, "dtype": "f64", "data": "synthetic",
        "config": {"workload": WORKLOAD, "parallelism": "host cores",
                   "sample": f"causal prefix of {n} tokens of one (batch, head) per step"},
        "cpu_baseline": {"value": round(value, 6), "unit": "TFLOP/s", "cores": os.cpu_count(),
                         "kind": "oracle", "sample": sample},
        "e2e": {"value": round(value, 6), "unit": "TFLOP/s", "h2d_bytes_per_step": 0,
                "d2h_bytes_per_step": 0},
    }), flush=True)


def run_ours(args, rank, world, local_rank):
    import torch
    import torch.distributed as dist

    torch.cuda.set_device(local_rank)
    if world > 1:
        dist.init_process_group("nccl", device_id=torch.device("cuda", local_rank))
    from exact_attention_41_gb300 import build as build_mod

    if rank == 0 or world == 1:
        build_mod.build()
    if world > 1:
        dist.barrier()
    from exact_attention_41_gb300 import libattn

    pk = peaks()
    stream = torch.cuda.current_stream()
    q, k, v, do = training_inputs()
    o = torch.empty_like(q)
    lse = torch.empty((B, HQ, S), device="cuda", dtype=torch.float32)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = libattn.bwd_workspace(q, k, False)
    ws_det = libattn.bwd_workspace(q, k, True)

    def fwd():
        libattn.fwd(q, k, v, causal=True, out=o, lse=lse)

    def bwd(det=False):
        libattn.bwd(q, k, v, o, lse, do, causal=True, deterministic=det,
                    workspace=ws_det if det else ws, dq=dq, dk=dk, dv=dv)

    def step():
        fwd()
        bwd()

    def fwd_bwd_into(xq, xk, xv, xdo, gq, gk, gv):
        libattn.fwd(xq, xk, xv, causal=True, out=o, lse=lse)
        libattn.bwd(xq, xk, xv, o, lse, xdo, causal=True, workspace=ws, dq=gq, dk=gk, dv=gv)

    for _ in range(max(3, args.warmup)):
        step()
    torch.cuda.synchronize()
    if world > 1:
        dist.barrier()
    n0 = libattn.launch_count()
    with ClockSampler(local_rank) as clk:
        ms = timed(step, args.steps, stream)
    launches = libattn.launch_count() - n0
    ms = max_over_ranks(ms, world, device="cuda")
    value = job_value(STEP_FLOPS, ms, world)

    extra_steps = max(5, min(args.steps, 20))
    ms_fwd = timed(fwd, extra_steps, stream)
    ms_bwd = timed(bwd, extra_steps, stream)
    ms_bwd_det = timed(lambda: bwd(True), extra_steps, stream)

    # FP8 forward (E4M3 copies of q, k, v; descales 1): the S products on the
    # FP8 tensor path, P V in bf16
    q8, k8, v8 = (x.to(torch.float8_e4m3fn) for x in (q, k, v))
    ws8 = torch.empty(libattn.lib().attn_fwd_fp8_workspace_size(B, S, HKV, D), device="cuda",
                      dtype=torch.uint8)

    def fwd8():
        libattn.fwd_fp8(q8, k8, v8, causal=True, out=o, lse=lse, workspace=ws8)

    fwd8()
    ms_fwd8 = timed(fwd8, extra_steps, stream)
    del q8, k8, v8, ws8

    # end to end through the public API from pinned host buffers
    ms_e2e, e2e_info = bench_e2e(libattn, (q, k, v, do), fwd_bwd_into, extra_steps, stream)
    out = None
    if rank == 0:
        peak_t = pk["bf16_tflops"]
        bwd_tflops = BWD_FLOPS / (ms_bwd * 1e-3) / 1e12
        fwd_tflops = FWD_FLOPS / (ms_fwd * 1e-3) / 1e12
        out = {
            "metric": METRIC, "value": round(value, 2), "unit": "TFLOP/s", "n_gpus": world,
            "steps": args.steps, "warmup": max(3, args.warmup), "ms_per_step": round(ms, 4),
            "higher_is_better": True, "scaling": "weak", "vs_baseline": None, "dtype": "bf16",
            "data": "synthetic: N(0,1) bf16 from torch's seeded CUDA generator",
            "config": {"workload": WORKLOAD, "global_batch": B * world, "seq_len": S,
                       "heads_q": HQ, "heads_kv": HKV, "head_dim": D,
                       "parallelism": f"replicas x{world} (no collective on the data path)",
                       "l2": "no flush: each step reads >= 896 MiB of inputs, above the 126 MB L2"},
            "frac_of_peak": round(value / world / pk["bf16_tflops_sustained"], 4),
            "peak_note": f"bf16 dense, {pk['source']} (sustained for the step, burst per kernel)",
            "tokens_per_s": round(world * B * S / (ms * 1e-3), 1),
            "fwd": {"ms": round(ms_fwd, 4), "tflops": round(fwd_tflops, 2),
                    "frac": round(fwd_tflops / peak_t, 4)},
            "bwd": {"ms": round(ms_bwd, 4), "tflops": round(bwd_tflops, 2),
                    "frac": round(bwd_tflops / peak_t, 4)},
            "fwd_fp8": {"ms": round(ms_fwd8, 4),
                        "tflops": round(FWD_FLOPS / (ms_fwd8 * 1e-3) / 1e12, 2),
                        "note": "E4M3 q,k,v; QK^T kind::f8f6f4, PV bf16; includes the V widening"},
            "bwd_deterministic": {"ms": round(ms_bwd_det, 4),
                                  "tflops": round(BWD_FLOPS / (ms_bwd_det * 1e-3) / 1e12, 2)},
            "roofline": {"bound": "tensor", "kernel": "backward (attn_bwd call)",
                         "achieved": round(bwd_tflops, 2), "peak": peak_t, "unit": "TFLOP/s",
                         "frac": round(bwd_tflops / peak_t, 4),
                         "traffic": traffic_for("bwd"), "traffic_note": TRAFFIC_NOTE,
                         "per_launch": "algorithmic bwd FLOPs 5.498e12 / CUDA-event time of "
                                       "one attn_bwd call"},
            "roofline_fwd": {"bound": "tensor", "kernel": "forward (attn_fwd call)",
                             "achieved": round(fwd_tflops, 2), "peak": peak_t, "unit": "TFLOP/s",
                             "frac": round(fwd_tflops / peak_t, 4), "traffic": traffic_for("fwd"),
                             "traffic_note": TRAFFIC_NOTE},
            "e2e": {"value": round(world * STEP_FLOPS / (ms_e2e * 1e-3) / 1e12, 2),
                    "unit": "TFLOP/s", "ms_per_step": round(ms_e2e, 4), **e2e_info},
            "gpu_launches": launches,
            "clocks": clk.summary(),
        }
    del ws_det
    if rank == 0 and not args.no_accuracy:
        out["accuracy"] = accuracy_sample(libattn, (q, k, v, do), o, lse, ws)
    if rank == 0 and not args.no_extras:
        del q, k, v, do, o, lse, dq, dk, dv, ws
        torch.cuda.empty_cache()
        out["varlen"] = bench_varlen(libattn, extra_steps, stream)
        torch.cuda.empty_cache()
        out["head_dims"] = bench_head_dims(libattn, extra_steps, stream)
        torch.cuda.empty_cache()
        for sq in (1, 4):
            r = bench_decode(libattn, extra_steps, stream, sq)
            r["frac_of_hbm"] = round(r["gbs"] / pk["hbm_gbs"], 4)
            out[f"decode_sq{sq}"] = r
            torch.cuda.empty_cache()
    if rank == 0 and not args.no_cpu_baseline:
        out["cpu_baseline"] = cpu_baseline_sample()
    if rank == 0:
        print(json.dumps(out), flush=True)
    if world > 1:
        dist.barrier()
        dist.destroy_process_group()


def run_profile_case(args):
    """One small, fixed case of one kernel family, for profiler captures
    (no timing, no JSON line); each is larger than L2 in its K/V or Q/dO
    streams and about 1 GB on the device at most:

    fwd / bwd   causal bf16 b=1 s=8192 hq=32 hkv=8 d=128 (`--deterministic`
                for that backward mode; `--head-dim` 64 or 256 keeps
                hq * d = 4096 and hkv = hq / 4, as the head-dim sweep does)
    decode      paged decode b=16, sq=s_new=4 (--decode-sq), hq=32 hkv=8, d=128
                (--head-dim 64 / 256 keep hq and hkv), caches U[1,32768]
                in 256-token pages (the workload's per-entry shape; 16 entries
                make several full waves of splits)
    varlen      the varlen workload (64 sequences U[100,4096], window (256,0),
                softcap 50), forward then backward
    paged       a serving step over a paged cache: the decode case's 16 caches
                (--head-dim as there) with one new token each but the first,
                which gets a chunk of 1024; appended, causal
    norm / norm_bwd
                per-head norm and rotation of the queries and keys of 16384
                tokens, or its gradient (--head-dim keeps hq * d = 4096)

    `--calls` calls (a warm-up and the one to capture), then the device
    error word is checked."""
    import torch

    from exact_attention_41_gb300 import build as build_mod

    build_mod.build()
    from exact_attention_41_gb300 import libattn
    from exact_attention_41_gb300 import synthetic as syn

    bf = syn.BF16
    if args.profile_case in ("fwd", "bwd"):
        d = args.head_dim
        b, s, hq = 1, S, HQ * D // d
        hkv = hq // 4
        q = syn.device_normal((b, s, hq, d), bf, 1)
        k = syn.device_normal((b, s, hkv, d), bf, 2)
        v = syn.device_normal((b, s, hkv, d), bf, 3)
        if args.profile_case == "fwd":
            for _ in range(args.calls):
                libattn.fwd(q, k, v, causal=True)
        else:
            do = syn.device_normal((b, s, hq, d), bf, 4)
            o, lse = libattn.fwd(q, k, v, causal=True)
            for _ in range(args.calls):
                libattn.bwd(q, k, v, o, lse, do, causal=True, deterministic=args.deterministic)
    elif args.profile_case == "varlen":
        lens = syn.varlen_lengths(7)
        cu = torch.from_numpy(syn.cu_seqlens(lens)).cuda()
        t, mx = int(lens.sum()), int(lens.max())
        q, k, v, do = (syn.device_normal((t, h, D), bf, 10 + i)
                       for i, h in enumerate((HQ, HKV, HKV, HQ)))
        kw = dict(causal=True, window=(256, 0), softcap=50.0)
        for _ in range(args.calls):
            o, lse = libattn.fwd_varlen(q, k, v, cu, cu, mx, mx, **kw)
        for _ in range(args.calls):
            libattn.bwd_varlen(q, k, v, o, lse, do, cu, cu, mx, mx,
                               deterministic=args.deterministic, **kw)
    elif args.profile_case in ("norm", "norm_bwd"):
        d = args.head_dim
        b, s, hq = 1, 16384, HQ * D // d
        q, k, gq, gk = (syn.device_normal((b, s, h, d), bf, 20 + i)
                        for i, h in enumerate((hq, hq // 4, hq, hq // 4)))
        wq, wk = (syn.device_normal((d,), bf, 24 + i) for i in range(2))
        ph = libattn.rope_phases([10000.0 ** (-2 * j / d) for j in range(d // 2)])
        kw = dict(phases=ph, q_weight=wq, k_weight=wk)
        for _ in range(args.calls):
            if args.profile_case == "norm":
                libattn.qk_norm_rope(q, k, **kw)
            else:
                libattn.qk_norm_rope_bwd(q, k, gq, gk, **kw)
    elif args.profile_case == "paged":
        b, chunk, page, d = 16, 1024, 256, args.head_dim
        seqlens, table, npages = syn.decode_layout(9, b, 32768, page, chunk)
        new = [chunk] + [1] * (b - 1)
        cu = torch.tensor([sum(new[:i]) for i in range(b + 1)], dtype=torch.int32).cuda()
        kc = syn.device_normal((npages, page, HKV, d), bf, 5)
        vc = syn.device_normal((npages, page, HKV, d), bf, 6)
        q = syn.device_normal((sum(new), HQ, d), bf, 7)
        sl, bt = torch.from_numpy(seqlens).cuda(), torch.from_numpy(table).cuda()
        for _ in range(args.calls):
            libattn.fwd_paged(q, kc, vc, cu, sl, block_table=bt, causal=True)
    else:
        b, sq, page, d = 16, args.decode_sq, 256, args.head_dim
        seqlens, table, npages = syn.decode_layout(9, b, 32768, page, sq)
        kc = syn.device_normal((npages, page, HKV, d), bf, 5)
        vc = syn.device_normal((npages, page, HKV, d), bf, 6)
        q = syn.device_normal((b, sq, HQ, d), bf, 7)
        kn = syn.device_normal((b, sq, HKV, d), bf, 8)
        vn = syn.device_normal((b, sq, HKV, d), bf, 9)
        sl = torch.from_numpy(seqlens).cuda()
        bt = torch.from_numpy(table).cuda()
        for _ in range(args.calls):
            libattn.fwd_kvcache(q, kc, vc, sl, k_new=kn, v_new=vn, block_table=bt, causal=True)
    torch.cuda.synchronize()
    st = libattn.device_error()
    print("profile case", args.profile_case, "done; device error", st, flush=True)
    sys.exit(0 if st == (0, 0) else 1)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--warmup", type=int, default=3)
    ap.add_argument("--impl", default="ours", choices=["ours", "reference"])
    ap.add_argument("--no-extras", action="store_true", help="skip varlen/decode lines")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--no-accuracy", action="store_true", help="skip the oracle error sample")
    ap.add_argument("--profile-case", choices=["fwd", "bwd", "decode", "varlen", "paged", "norm", "norm_bwd"],
                    help="run one small fixed case for a profiler capture and exit")
    ap.add_argument("--calls", type=int, default=2, help="calls of --profile-case")
    ap.add_argument("--deterministic", action="store_true", help="--profile-case bwd mode")
    ap.add_argument("--decode-sq", type=int, default=4, help="--profile-case decode: sq = s_new")
    ap.add_argument("--head-dim", type=int, default=128, choices=[64, 128, 256],
                    help="--profile-case fwd/bwd: head dim (hq = 4096 / d), norm too; decode/paged: head dim")
    args = ap.parse_args()
    rank = int(os.environ.get("RANK", "0"))
    world = int(os.environ.get("WORLD_SIZE", "1"))
    local_rank = int(os.environ.get("LOCAL_RANK", "0"))
    if args.profile_case:
        run_profile_case(args)
        return
    if args.impl == "reference":
        run_reference(args, rank)
        return
    run_ours(args, rank, world, local_rank)


if __name__ == "__main__":
    main()
