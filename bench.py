#!/usr/bin/env python3
"""Benchmark of the SVDQuant W4A4 linear on one MI355X.

Workload (one "step" = the whole hot path of one layer over one batch):
the FLUX-like MLP fc1 linear, 4608 tokens x 3072 -> 12288, rank 32, INT4
group 64, GELU-tanh epilogue, bias:  svdq_quantize_act (smoothing + INT4
quantization + rank-32 down projection) followed by svdq_w4a4_linear (4-bit
product + low-rank up projection + bias + GELU + bf16 store).  Inputs are
seeded synthetic tensors already resident in HBM; the weights are packed once
on the host before timing.  Several input/output buffer sets (> 256 MB in all)
rotate so the 256 MB last-level cache cannot hold a step's working set.

value = 2 M N K / (time per step), in TOPS (tera integer ops of the 4-bit
product per second).  The JSON line also carries the roofline of the dominant
kernel (svdq_w4a4_linear vs the dense int8 matrix peak), the activation
kernel's HBM rate, and the fp64 CPU oracle timed on a bounded row sample.
"""
from __future__ import annotations

import argparse
import json
import os
import sys
import time

ROOT = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, ROOT)

import numpy as np  # noqa: E402

PEAK_INT8_TOPS = 5000.0     # MI355X dense int8 matrix peak, 5.0 POP/s
PEAK_FP4_TFLOPS = 10100.0   # MI355X dense MXFP4 matrix peak, 10.1 PFLOP/s
PEAK_BF16_TFLOPS = 2500.0   # MI355X dense bf16 matrix peak, 2.5 PFLOP/s
PEAK_HBM_GBS = 8000.0       # MI355X HBM3E, 8 TB/s
NO_CLOCK = False

# HBM traffic per launch of a workload's kernel, from two rocprofv3 --pmc runs
# (FETCH_SIZE, then WRITE_SIZE) of this script, each divided by what the same
# counter reads for a plain 512 MiB copy (--copy-calibration).  An entry is
# only reported while the kernel source, with the device code that it includes,
# still hashes to the value it was measured on; otherwise traffic is null.
TRAFFIC = {
    # FETCH_SIZE 73572.1 KiB / 0.50002 + WRITE_SIZE 110601.9 KiB / 1.00000 (per dispatch)
    "fc1": {"source": "w4a4_gemm.hip", "source_sha": "783bff217a40e369", "bytes": 263925397},
    # FETCH_SIZE 70190.8 KiB / 0.50002 + WRITE_SIZE 110600.1 KiB / 1.00000
    "mx_fc1": {"source": "w4a4_gemm.hip", "source_sha": "783bff217a40e369", "bytes": 256998955},
    # FETCH_SIZE 15680.0 KiB / 0.50002 + WRITE_SIZE 36.0 KiB / 1.00000
    "awq_mod": {"source": "awq_gemv.hip", "source_sha": "8e9f775e255a96a4", "bytes": 32148095},
    # FETCH_SIZE 197077.9 KiB / 0.50002 + WRITE_SIZE 110597.2 KiB / 1.00000
    "nf4_fc1": {"source": "nf4_gemm.hip", "source_sha": "9324426f1560d454", "bytes": 516849367},
}


def measured_traffic(workload):
    """HBM bytes per launch of the named workload's kernel (the synth spec
    name: a table entry covers that shape only) from the table above, or None
    once the kernel source no longer hashes to the value the counters were
    taken on."""
    t = TRAFFIC.get(workload)
    if t is None or t["source_sha"] != _source_sha(t["source"]):
        return None
    return t["bytes"]


def _source_sha(name):
    """Hash of a kernel source and of the device code in the headers that it
    includes, without comments and blanks."""
    import hashlib
    import re
    csrc = os.path.join(ROOT, "w4a4_rank_corrected_quantize_amd", "csrc")
    todo, seen, digest = [name], set(), hashlib.sha256()
    while todo:
        path = os.path.join(csrc, todo.pop(0))
        if path in seen or not os.path.exists(path):      # include/svdq.h: declarations
            continue
        seen.add(path)
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        todo += re.findall(r'#include "([^"]+)"', text)
        if path.endswith(".hip") or "__device__" in text:
            digest.update("".join(text.split()).encode())
    return digest.hexdigest()[:16]


def copy_calibration(mib):
    """A plain device-to-device copy of known size, for scaling HBM counters."""
    import torch
    n = mib << 20
    src = torch.empty(n, dtype=torch.uint8, device="cuda").fill_(1)
    dst = torch.empty_like(src)
    torch.cuda.synchronize()
    for _ in range(3):
        dst.copy_(src)
    torch.cuda.synchronize()
    print(json.dumps({"copy_calibration_bytes_read": n, "bytes_written": n, "launches": 3}), flush=True)


def host_info():
    """The CPU model and the hardware threads this process may use (the CPU
    baseline's `cores` is what the oracle actually ran on)."""
    model = None
    try:
        with open("/proc/cpuinfo") as f:
            for ln in f:
                if ln.startswith("model name"):
                    model = ln.split(":", 1)[1].strip()
                    break
    except OSError:
        pass
    return {"cpu_model": model, "cpu_threads": len(os.sched_getaffinity(0))}


def gpu_clock(torch, step, ms_per_step, seconds=1.0, period=0.05, what="steps"):
    """The GFX clock while the step runs back to back: after the timed region
    the step is enqueued for about `seconds` while a second thread reads the
    clock that amd-smi reports (torch.cuda.clock_rate) every `period` s.  The
    samples of the first 0.2 s are dropped (the reading averages over a window
    that can reach back into the gap before the run).  None where amd-smi is
    unavailable."""
    import threading
    if NO_CLOCK:
        return None
    try:
        torch.cuda.clock_rate(0)
    except Exception:
        return None
    samples, stop = [], threading.Event()

    def sample():
        t0 = time.time()
        while not stop.is_set():
            try:
                mhz = float(torch.cuda.clock_rate(0))
            except Exception:
                return
            if time.time() - t0 > 0.2 and mhz > 0:
                samples.append(mhz)
            stop.wait(period)

    n = min(20000, max(1, int(seconds * 1e3 / max(ms_per_step, 1e-3))))
    torch.cuda.synchronize()
    th = threading.Thread(target=sample, daemon=True)
    th.start()
    for i in range(n):
        step(i)
    torch.cuda.synchronize()
    stop.set()
    th.join()
    if not samples:
        return None
    return {"source": f"amd-smi GFX clock (the SMU's reported value, not a shader-cycle count), sampled every "
                      f"{int(period * 1e3)} ms while {n} more {what} ran back to back after the timed region",
            "median_MHz": float(np.median(samples)), "min_MHz": min(samples), "max_MHz": max(samples),
            "samples": len(samples)}


def k1_bytes(M, K, r, prec):
    scales = (M * K // 64) * 4 if prec == 0 else M * K // 32
    return 2 * M * K + M * K // 2 + scales + 4 * M * r + 4 * K + 2 * r * K


def k2_bytes(M, N, K, r, prec, bias=True):
    scales = lambda rows: (rows * K // 64) * 4 if prec == 0 else rows * K // 32  # noqa: E731
    return (M * K // 2 + scales(M) + 4 * M * r + N * K // 2 + scales(N) + 2 * N * r
            + (2 * N if bias else 0) + 2 * M * N)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--gpus", type=int, default=1)
    # the clock settles only after ~30 ms of back-to-back launches (the
    # linear's time falls from ~410 to ~320 us over its first ~90 launches),
    # so the default warm-up covers that ramp
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--warmup", type=int, default=200)
    ap.add_argument("--prec", choices=["int4", "mxfp4"], default="int4")
    ap.add_argument("--layer", choices=["fc1", "qkv", "fc2", "mlp", "awq", "qkvnorm", "nf4_fc1", "nf4_qkv"],
                    default="fc1",
                    help="fc1 is the headline workload; fc2 takes fc1's output (computed on the GPU); "
                         "mlp times fc1 -> fc2 with fc2's activation step fused into fc1's epilogue, "
                         "next to the unfused pair; awq times the weight-only AWQ W4A16 modulation layer; "
                         "qkvnorm is qkv with the Q/K RMS-norm and rotary embedding fused into the epilogue; "
                         "nf4_fc1 / nf4_qkv time the weight-only NF4 W4A16 comparison path on those shapes")
    ap.add_argument("--copy-calibration", type=int, metavar="MIB", default=0,
                    help="only run a plain copy of MIB MiB (to scale the HBM byte counters)")
    ap.add_argument("--sets", type=int, default=0,
                    help="rotating buffer sets (default 3; 12 for awq, whose 32 MB of weights per set "
                         "would otherwise stay in the 256 MB last-level cache)")
    ap.add_argument("--tokens", type=int, choices=[4608, 1024], default=4608,
                    help="1024: the MXFP4 linears of a 512 x 512 image (--prec mxfp4, fc1 / qkv / fc2)")
    ap.add_argument("--launch", choices=["eager", "graph"], default=None,
                    help="graph: capture the timed steps (and each kernel's launches) in HIP graphs and time their "
                         "replays, so host launch gaps do not count; default graph for --tokens 1024 (kernels of "
                         "10-40 us that the host cannot keep fed), eager otherwise")
    ap.add_argument("--splitk", action="store_true",
                    help="time svdq_w4a4_linear_splitk (K split across work items when the tiles cannot fill "
                         "the chip; the workspace is allocated before the timed region)")
    ap.add_argument("--no-cpu-baseline", action="store_true")
    ap.add_argument("--settle-ms", type=float, default=100.0,
                    help="untimed steps for at least this long before the warm-up, so that the GPU clock has "
                         "left its idle level whatever --warmup is (0: none)")
    ap.add_argument("--no-clock", action="store_true",
                    help="skip the clock sampling after the timed region (under a counter profiler)")
    ap.add_argument("--cpu-seconds", type=float, default=15.0, help="target oracle sample time")
    args = ap.parse_args()
    global NO_CLOCK
    NO_CLOCK = args.no_clock
    if args.gpus != 1 or int(os.environ.get("WORLD_SIZE", "1")) != 1:
        print("bench.py measures one GPU only: the layer runs on a single MI355X and there is "
              "no multi-GPU path; run it with --gpus 1.", file=sys.stderr)
        sys.exit(2)

    import torch

    if args.copy_calibration:
        torch.cuda.set_device(0)
        copy_calibration(args.copy_calibration)
        return

    import w4a4_rank_corrected_quantize_amd as svdq
    from w4a4_rank_corrected_quantize_amd import synth

    torch.cuda.set_device(0)
    svdq.check_device()
    if args.layer == "mlp":
        mlp_main(args, torch, svdq, synth)
        return
    if args.layer == "awq":
        awq_main(args, torch, svdq, synth)
        return
    if args.layer.startswith("nf4_"):
        nf4_main(args, torch, svdq, synth)
        return
    if not args.sets:
        args.sets = 3
    prec = svdq.INT4 if args.prec == "int4" else svdq.MXFP4
    qkvnorm = args.layer == "qkvnorm"
    if args.tokens != 4608 and (prec != svdq.MXFP4 or args.layer not in ("fc1", "qkv", "fc2")):
        print("--tokens 1024 is the MXFP4 fc1 / qkv / fc2 workload", file=sys.stderr)
        sys.exit(2)
    pre = "" if prec == svdq.INT4 else ("mx_" if args.tokens == 4608 else "mx1k_")
    spec = synth.SPECS[pre + ("qkv" if qkvnorm else args.layer)]
    M, K, N, r = spec.M, spec.K, spec.N, svdq.RANK
    X_bits = None
    if args.layer == "fc2":
        # fc2's input is fc1's bf16 output: run fc1 once on the GPU to make it
        f1 = synth.SPECS[pre + "fc1"]
        print(f"[bench] making fc2's input with {f1.name} on the GPU", file=sys.stderr, flush=True)
        L1 = synth.make_layer(f1)
        d1 = svdq.to_device(svdq.pack_weights(L1["W"], L1["act_absmax"], prec=prec))
        xq1, xs1, h1 = svdq.quantize_act(svdq.bf16_tensor(L1["X"]), d1["smooth"], d1["down"], prec)
        Y1 = svdq.w4a4_linear(xq1, xs1, h1, d1["wq"], d1["wscale"], d1["up"], svdq.bf16_tensor(L1["bias"]),
                              prec, svdq.EPI_GELU_TANH)
        X_bits = svdq.bf16_bits(Y1)
        del L1, d1, xq1, xs1, h1, Y1
    print(f"[bench] generating {spec.name} {M}x{K}->{N} and packing on the host", file=sys.stderr,
          flush=True)
    L = synth.make_layer(spec, X_bits=X_bits)
    epi = svdq.EPI_GELU_TANH if spec.gelu else svdq.EPI_NONE
    t0 = time.time()
    p = svdq.pack_weights(L["W"], L["act_absmax"], prec=prec)
    pack_s = time.time() - t0
    g = svdq.group_of(prec)
    sdt = torch.float32 if prec == svdq.INT4 else torch.uint8

    sets = []
    for i in range(args.sets):
        d = svdq.to_device(p)
        sets.append(dict(
            X=svdq.bf16_tensor(L["X"]), smooth=d["smooth"], down=d["down"], up=d["up"], wq=d["wq"],
            wscale=d["wscale"], bias=None if L["bias"] is None else svdq.bf16_tensor(L["bias"]),
            xq=torch.empty((M, K // 2), dtype=torch.uint8, device="cuda"),
            xscale=torch.empty((M, K // g), dtype=sdt, device="cuda"),
            h=torch.empty((M, r), dtype=torch.float32, device="cuda"),
            Y=torch.empty((M, N), dtype=torch.bfloat16, device="cuda")))
    work = None
    if args.splitk:
        if qkvnorm:
            print("--splitk does not apply to --layer qkvnorm", file=sys.stderr)
            sys.exit(2)
        nb = svdq.linear_splitk_workspace_bytes(M, N, K, prec)
        work = torch.empty(max(nb // 4, 1), dtype=torch.float32, device="cuda")
        print(f"[bench] split-K workspace {nb / 1e6:.1f} MB", file=sys.stderr, flush=True)
    ws_mb = sum(t.numel() * t.element_size() for t in sets[0].values() if t is not None) / 1e6
    if qkvnorm:
        rc, rs = synth.gen_rope(M)
        qkn = dict(nq=svdq.bf16_tensor(synth.gen_qk_norm(spec.config_id, 10)),
                   nk=svdq.bf16_tensor(synth.gen_qk_norm(spec.config_id, 11)),
                   c=torch.from_numpy(rc).cuda(), s=torch.from_numpy(rs).cuda())

    def k1(b):
        svdq.quantize_act(b["X"], b["smooth"], b["down"], prec, xq=b["xq"], xscale=b["xscale"], h=b["h"])

    def k2(b):
        if qkvnorm:
            svdq.w4a4_linear_qkv_norm_rope(b["xq"], b["xscale"], b["h"], b["wq"], b["wscale"], b["up"], b["bias"],
                                           qkn["nq"], qkn["nk"], 1e-6, qkn["c"], qkn["s"], prec, Y=b["Y"])
            return
        if work is not None:
            svdq.w4a4_linear_splitk(b["xq"], b["xscale"], b["h"], b["wq"], b["wscale"], b["up"], b["bias"], prec,
                                    epi, Y=b["Y"], work=work)
            return
        svdq.w4a4_linear(b["xq"], b["xscale"], b["h"], b["wq"], b["wscale"], b["up"], b["bias"], prec,
                         epi, Y=b["Y"])

    settled = settle(torch, lambda i: (k1(sets[i % len(sets)]), k2(sets[i % len(sets)])), args.settle_ms)
    for i in range(args.warmup):
        k1(sets[i % len(sets)])
        k2(sets[i % len(sets)])
    torch.cuda.synchronize()
    print(f"[bench] settled ({settled} steps), warmup done ({args.warmup} steps); timing {args.steps} steps",
          file=sys.stderr, flush=True)

    def ev():
        return torch.cuda.Event(enable_timing=True)

    launch = args.launch or ("graph" if args.tokens == 1024 else "eager")
    if launch == "graph":
        ms_per_step, k1_ms, k2_ms, g_step = graph_times(torch, sets, k1, k2, args.steps)
    else:
        # 1) the timed region: K whole steps, events only at its ends
        start, stop = ev(), ev()
        torch.cuda.synchronize()
        start.record()
        for i in range(args.steps):
            k1(sets[i % len(sets)])
            k2(sets[i % len(sets)])
        stop.record()
        torch.cuda.synchronize()
        total_ms = start.elapsed_time(stop)
        ms_per_step = total_ms / args.steps

        # 2) the same K steps again, with event pairs around each launch (on
        #    torch's current stream, where both calls enqueue).  The linear's
        #    times agree with rocprofv3's kernel trace; the activation kernel
        #    is short enough (~20 us) that an event pair adds a few us to it.
        evs = [(ev(), ev(), ev()) for _ in range(args.steps)]
        torch.cuda.synchronize()
        for i in range(args.steps):
            evs[i][0].record()
            k1(sets[i % len(sets)])
            evs[i][1].record()
            k2(sets[i % len(sets)])
            evs[i][2].record()
        torch.cuda.synchronize()
        k1_ms = float(np.mean([e[0].elapsed_time(e[1]) for e in evs]))
        k2_ms = float(np.mean([e[1].elapsed_time(e[2]) for e in evs]))

    ops = 2.0 * M * N * K
    value = ops / (ms_per_step * 1e-3) / 1e12
    k2_tops = ops / (k2_ms * 1e-3) / 1e12
    ref = library_reference(torch, M, N, K)
    peak = PEAK_INT8_TOPS if prec == svdq.INT4 else PEAK_FP4_TFLOPS
    k1_gbs = k1_bytes(M, K, r, prec) / (k1_ms * 1e-3) / 1e9
    k2_gbs = k2_bytes(M, N, K, r, prec, bias=L["bias"] is not None) / (k2_ms * 1e-3) / 1e9
    traffic = None if qkvnorm else measured_traffic(spec.name)

    if launch == "graph":
        clock = gpu_clock(torch, lambda i: g_step.replay(), ms_per_step * args.steps,
                          what=f"replays of the {args.steps}-step graph")
    else:
        clock = gpu_clock(torch, lambda i: (k1(sets[i % len(sets)]), k2(sets[i % len(sets)])), ms_per_step)
    cpu = None
    if not args.no_cpu_baseline:
        from oracle import oracle as O
        print("[bench] timing the CPU oracle on a row sample", file=sys.stderr, flush=True)
        # a 64-row probe sizes the sample (a smaller one is dominated by the
        # per-call cost and undersizes it)
        rows = min(M, 64)
        t0 = time.time()
        xq, xs, h = O.quant_act(L["X"][:rows], p["smooth"], p["down"], prec)
        O.linear(xq, xs, h, p["wq"], p["wscale"], p["up"], L["bias"], prec, gelu=spec.gelu)
        probe = max(time.time() - t0, 1e-3)
        rows = int(min(M, max(8, rows * args.cpu_seconds / probe)))
        t0 = time.time()
        xq, xs, h = O.quant_act(L["X"][:rows], p["smooth"], p["down"], prec)
        yl = O.linear(xq, xs, h, p["wq"], p["wscale"], p["up"], L["bias"], prec, gelu=spec.gelu)
        if qkvnorm:
            O.qkv_norm_rope(yl, synth.gen_qk_norm(spec.config_id, 10), synth.gen_qk_norm(spec.config_id, 11), 1e-6,
                            rc[:rows], rs[:rows])
        t_cpu = time.time() - t0
        cpu = {"value": round(2.0 * rows * N * K / t_cpu / 1e12, 6), "unit": "TOPS", "cores": O.num_threads(),
               "kind": "oracle",
               "sample": f"{rows} of {M} token rows of the same layer (activation step + linear), "
                         f"{t_cpu:.1f} s"}

    headline = prec == svdq.INT4 and spec.name == "fc1" and not qkvnorm and work is None
    metric = ("W4A4 linear TOPS & % int8-MFMA peak at M=4608,K=3072,N=12288 (r=32)" if headline else
              f"W4A4 linear {'TOPS' if prec == svdq.INT4 else 'TFLOP/s'} & % "
              f"{'int8' if prec == svdq.INT4 else 'fp4'}-MFMA peak at M={M},K={K},N={N} (r={r})"
              f"{', Q/K norm + rotary epilogue' if qkvnorm else ''}{', split K' if work is not None else ''}")
    line = {
        "metric": metric,
        "value": round(value, 2),
        "unit": "TOPS" if prec == svdq.INT4 else "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "settle": {"ms": args.settle_ms, "steps": settled},
        "ms_per_step": round(ms_per_step, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int4 codes as exact fp8 E4M3 subnormals on the fp8 matrix cores (exact per-group partials); "
                 "group scale sx*sw from a bf16 hi/lo matrix product (~2^-16 relative), one fp32 fma per group"
        if prec == svdq.INT4
        else "mxfp4 (e2m1 x e2m1, e8m0 scales) on the scaled fp4 matrix cores, fp32 accumulation",
        "data": "synthetic (seeded Student-t activations with outlier channels, N(0,0.02^2) weights)",
        "config": {"workload": f"{spec.name}: {M} tokens x {K} -> {N}, rank {r}, "
                               f"{'INT4 g64' if prec == svdq.INT4 else 'MXFP4 g32'}, bias"
                               f"{', GELU-tanh' if spec.gelu else ''}"
                               f"{', Q/K RMS-norm + rotary embedding in the epilogue' if qkvnorm else ''}; "
                               "step = svdq_quantize_act + "
                               f"{'svdq_w4a4_linear_qkv_norm_rope' if qkvnorm else 'svdq_w4a4_linear'}",
                   "M": M, "K": K, "N": N, "rank": r, "buffer_sets": len(sets),
                   "working_set_MB_per_set": round(ws_mb, 1), "launch": launch},
        "roofline": {"bound": "mfma", "kernel": ("svdq_w4a4_linear_qkv_norm_rope" if qkvnorm else
                                                  "svdq_w4a4_linear_splitk (both kernels)" if work is not None
                                                  else "svdq_w4a4_linear"),
                     "achieved": round(k2_tops, 2), "peak": peak,
                     "unit": "TFLOP/s", "frac": round(k2_tops / peak, 4), "traffic": traffic,
                     "avg_ms": round(k2_ms, 5)},
        "activation_kernel": {"kernel": "svdq_quantize_act", "bound": "hbm", "avg_ms": round(k1_ms, 5),
                              "achieved_GBs": round(k1_gbs, 1), "peak_GBs": PEAK_HBM_GBS,
                              "frac": round(k1_gbs / PEAK_HBM_GBS, 4),
                              "algorithmic_bytes": k1_bytes(M, K, r, prec)},
        "linear_kernel_GBs": round(k2_gbs, 1),
        "matrix_core_reference": ref,
        "host_pack_s": round(pack_s, 2),
        "gpu_clock": clock,
        "host": host_info(),
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


def settle(torch, step, ms):
    """Runs the step back to back, untimed, for at least `ms` of wall time
    before the warm-up steps.  The GFX clock of an idle MI355X takes ~30 ms
    of back-to-back work to reach its sustained level (the linear's time
    falls from ~410 to ~320 us over its first ~90 launches), so a short
    warm-up would otherwise time part of the ramp.  Returns the number of
    steps run."""
    if ms <= 0:
        return 0
    n = 0
    t0 = time.time()
    while (time.time() - t0) * 1e3 < ms:
        for _ in range(4):
            step(n)
            n += 1
        torch.cuda.synchronize()
    return n


def graph_times(torch, sets, k1, k2, steps):
    """Per-step, activation-kernel and linear times from HIP-graph replays:
    one graph of `steps` whole steps, one of `steps` activation launches and
    one of `steps` linear launches, each replayed once between two events.
    The step graph's outputs are checked against eager launches (three
    replays, the outputs cleared in between) before anything is timed."""
    n = len(sets)

    def capture(body):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for i in range(steps):
                body(sets[i % n])
        torch.cuda.synchronize()
        return g

    g_step = capture(lambda b: (k1(b), k2(b)))
    g_k1 = capture(k1)
    g_k2 = capture(k2)
    ref = []
    for b in sets[:min(n, steps)]:
        k1(b)
        k2(b)
        ref.append(b["Y"].clone())
    torch.cuda.synchronize()
    for _ in range(3):
        for b in sets:
            b["Y"].zero_()
        g_step.replay()
        torch.cuda.synchronize()
        for b, y in zip(sets, ref):
            if not torch.equal(b["Y"], y):
                raise RuntimeError("graph replay differs from the eager launches")

    def timed(g):
        g.replay()                       # once untimed
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        e0.record()
        g.replay()
        e1.record()
        torch.cuda.synchronize()
        return e0.elapsed_time(e1) / steps

    return timed(g_step), timed(g_k1), timed(g_k2), g_step


def library_reference(torch, M, N, K, reps=20):
    """Dense GEMMs of the same shape through torch (hipBLASLt): fp8 e4m3 with
    per-tensor scales and bf16.  They are what the matrix cores reach here on
    a plain contraction: a measured ceiling for the same M, N, K, next to the
    nominal peak.  None where torch lacks the op."""
    out = {"kind": "torch._scaled_mm fp8 e4m3 (per-tensor scales) and torch.matmul bf16, "
                   f"{M} x {K} -> {N}, no quantization groups, no epilogue"}
    a = torch.randn(M, K, device="cuda")
    b = torch.randn(N, K, device="cuda")

    def rate(fn):
        for _ in range(3):
            fn()
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for _ in range(reps):
            fn()
        e1.record()
        torch.cuda.synchronize()
        return round(2.0 * M * N * K / (e0.elapsed_time(e1) / reps * 1e-3) / 1e12, 1)
    try:
        a8, b8 = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
        one = torch.tensor(1.0, device="cuda")
        out["fp8_tflops"] = rate(lambda: torch._scaled_mm(a8, b8.t(), scale_a=one, scale_b=one,
                                                          out_dtype=torch.bfloat16))
    except Exception:
        out["fp8_tflops"] = None
    a16, b16 = a.to(torch.bfloat16), b.to(torch.bfloat16)
    out["bf16_tflops"] = rate(lambda: a16 @ b16.t())
    return out


def awq_bytes(M, N, K, bias=True):
    return N * K // 2 + (N * K // 64) * 4 + 2 * M * K + 2 * M * N + (2 * N if bias else 0)


def awq_main(args, torch, svdq, synth):
    """The weight-only AWQ W4A16 layer (INT4 g64 weights, bf16 activations)
    at the modulation shape: HBM-bound on the weight stream."""
    spec = synth.SPECS["awq_mod"]
    M, K, N = spec.M, spec.K, spec.N
    nsets = args.sets or 12
    print(f"[bench] generating {spec.name} {M}x{K}->{N} and packing on the host", file=sys.stderr, flush=True)
    L = synth.make_layer(spec)
    t0 = time.time()
    wq, ws = svdq.awq_pack_weights(L["W"])
    pack_s = time.time() - t0
    sets = []
    for i in range(nsets):
        sets.append(dict(X=svdq.bf16_tensor(L["X"]), wq=torch.from_numpy(wq).cuda(),
                         ws=torch.from_numpy(ws).cuda(), b=svdq.bf16_tensor(L["bias"]),
                         Y=torch.empty((M, N), dtype=torch.bfloat16, device="cuda")))

    def step(b):
        svdq.awq_w4a16_linear(b["X"], b["wq"], b["ws"], b["b"], Y=b["Y"])

    for i in range(args.warmup):
        step(sets[i % nsets])
    torch.cuda.synchronize()
    # A 12 us kernel outruns the host's launches (~25 us each through the
    # binding), so the K timed steps are captured once in a HIP graph and
    # replayed: the timed region then holds the GPU's work, not host gaps.
    # Each replay's outputs are checked against an eager step first.
    launch = "hip graph"
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for i in range(args.steps):
                step(sets[i % nsets])
        torch.cuda.synchronize()
        ref = []
        for b in sets[:min(nsets, args.steps)]:
            step(b)
            ref.append(b["Y"].clone())
        torch.cuda.synchronize()
        for _ in range(3):
            for b in sets:
                b["Y"].zero_()
            graph.replay()
            torch.cuda.synchronize()
            for b, r in zip(sets, ref):
                if not torch.equal(b["Y"], r):
                    raise RuntimeError("graph replay differs from the eager launch")
    except Exception as e:      # report, and time the launches eagerly instead
        print(f"[bench] graph capture not used ({e}); timing eager launches", file=sys.stderr, flush=True)
        graph, launch = None, "eager"
    print(f"[bench] warmup done ({args.warmup} steps); timing {args.steps} steps ({launch})", file=sys.stderr,
          flush=True)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    if graph is not None:
        graph.replay()
    else:
        for i in range(args.steps):
            step(sets[i % nsets])
    stop.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop) / args.steps
    nbytes = awq_bytes(M, N, K)
    if graph is not None:   # eager launches leave the GPU idle between them (host-bound)
        clock = gpu_clock(torch, lambda i: graph.replay(), ms * args.steps,
                          what=f"replays of the {args.steps}-launch graph")
    else:
        clock = gpu_clock(torch, lambda i: step(sets[i % nsets]), ms)
    gbs = nbytes / (ms * 1e-3) / 1e9
    cpu = None
    if not args.no_cpu_baseline:
        from oracle import oracle as O
        print("[bench] timing the CPU oracle on the same layer", file=sys.stderr, flush=True)
        t0 = time.time()
        O.awq_linear(L["X"], wq, ws, L["bias"])
        t_cpu = time.time() - t0
        cpu = {"value": round(nbytes / t_cpu / 1e9, 3), "unit": "GB/s", "cores": 1, "kind": "oracle",
               "sample": f"the whole layer ({M} x {K} -> {N}) once, {t_cpu:.1f} s (one thread: the "
                         "oracle distributes rows of X, and there is one)"}
    line = {
        "metric": "AWQ W4A16 modulation linear, algorithmic GB/s of the weight stream",
        "value": round(gbs, 1),
        "unit": "GB/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int4 weights (g64, fp32 scales) x bf16 activations on the bf16 matrix cores, fp32 accumulation",
        "data": "synthetic (seeded N(0,1) activations, N(0,0.02^2) weights, N(0,0.01^2) bias)",
        "config": {"workload": f"{spec.name}: {M} x {K} -> {N}, INT4 g64 weight-only, bias; "
                               "step = svdq_awq_w4a16_linear",
                   "M": M, "K": K, "N": N, "buffer_sets": nsets,
                   "weights_MB_per_set": round((wq.nbytes + ws.nbytes) / 1e6, 1), "launch": launch},
        "roofline": {"bound": "hbm", "kernel": "svdq_awq_w4a16_linear", "achieved": round(gbs, 1),
                     "peak": PEAK_HBM_GBS, "unit": "GB/s", "frac": round(gbs / PEAK_HBM_GBS, 4),
                     "traffic": measured_traffic(spec.name), "avg_ms": round(ms, 5),
                     "algorithmic_bytes": nbytes},
        "host_pack_s": round(pack_s, 2),
        "gpu_clock": clock,
        "host": host_info(),
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


def nf4_bytes(M, N, K):
    nb = N * (K // 64)
    return 2 * M * K + N * K // 2 + nb + 4 * ((nb + 255) // 256) + 2 * M * N


def nf4_main(args, torch, svdq, synth):
    """The weight-only NF4 W4A16 comparison path (bf16 activations, NF4
    weights with double-quantized statistics, dequantized inside the bf16
    matrix-core GEMM) on the QKV or fc1 shape at 4608 tokens."""
    spec = synth.SPECS[args.layer]
    M, K, N = spec.M, spec.K, spec.N
    nsets = args.sets or 3
    print(f"[bench] generating {spec.name} {M}x{K}->{N} and packing on the host", file=sys.stderr, flush=True)
    L = synth.make_layer(spec)
    t0 = time.time()
    wq, qabs, chunk = svdq.nf4_pack_weights(L["W"])
    pack_s = time.time() - t0
    sets = [dict(X=svdq.bf16_tensor(L["X"]), wq=torch.from_numpy(wq).cuda(), qa=torch.from_numpy(qabs).cuda(),
                 ch=torch.from_numpy(chunk).cuda(), Y=torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
            for _ in range(nsets)]

    def step(b):
        svdq.nf4_w4a16_linear(b["X"], b["wq"], b["qa"], b["ch"], None, Y=b["Y"])

    settled = settle(torch, lambda i: step(sets[i % nsets]), args.settle_ms)
    for i in range(args.warmup):
        step(sets[i % nsets])
    torch.cuda.synchronize()
    print(f"[bench] settled ({settled} steps), warmup done ({args.warmup} steps); timing {args.steps} steps",
          file=sys.stderr, flush=True)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for i in range(args.steps):
        step(sets[i % nsets])
    stop.record()
    torch.cuda.synchronize()
    ms = start.elapsed_time(stop) / args.steps
    flops = 2.0 * M * N * K
    clock = gpu_clock(torch, lambda i: step(sets[i % nsets]), ms)
    tflops = flops / (ms * 1e-3) / 1e12
    ref = library_reference(torch, M, N, K)
    cpu = None
    if not args.no_cpu_baseline:
        from oracle import oracle as O
        print("[bench] timing the CPU oracle on a row sample", file=sys.stderr, flush=True)
        oq, oa, oc = O.nf4_pack(L["W"])
        rows = 64
        t0 = time.time()
        O.nf4_linear(L["X"], oq, oa, oc, None, rows=np.arange(rows, dtype=np.int32))
        probe = max(time.time() - t0, 1e-3)
        rows = int(min(M, max(8, rows * args.cpu_seconds / probe)))
        t0 = time.time()
        O.nf4_linear(L["X"], oq, oa, oc, None, rows=np.arange(rows, dtype=np.int32))
        t_cpu = time.time() - t0
        cpu = {"value": round(2.0 * rows * N * K / t_cpu / 1e12, 6), "unit": "TFLOP/s", "cores": O.num_threads(),
               "kind": "oracle", "sample": f"{rows} of {M} token rows of the same layer, {t_cpu:.1f} s"}
    line = {
        "metric": "NF4 W4A16 linear TFLOP/s & % bf16-MFMA peak (weight-only comparison path)",
        "value": round(tflops, 2),
        "unit": "TFLOP/s",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "settle": {"ms": args.settle_ms, "steps": settled},
        "ms_per_step": round(ms, 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "nf4 weights (64-blocks, 8-bit double-quantized statistics per 256 blocks) dequantized to bf16 "
                 "in the kernel x bf16 activations on the bf16 matrix cores, fp32 accumulation",
        "data": "synthetic (seeded N(0,1) activations, N(0,0.02^2) weights)",
        "config": {"workload": f"{spec.name}: {M} tokens x {K} -> {N}, NF4 weight-only, no bias; "
                               "step = svdq_nf4_w4a16_linear",
                   "M": M, "K": K, "N": N, "buffer_sets": nsets},
        "roofline": {"bound": "mfma", "kernel": "svdq_nf4_w4a16_linear", "achieved": round(tflops, 2),
                     "peak": PEAK_BF16_TFLOPS, "unit": "TFLOP/s", "frac": round(tflops / PEAK_BF16_TFLOPS, 4),
                     "traffic": measured_traffic(spec.name), "avg_ms": round(ms, 5),
                     "algorithmic_bytes": nf4_bytes(M, N, K)},
        "matrix_core_reference": ref,
        "host_pack_s": round(pack_s, 2),
        "gpu_clock": clock,
        "host": host_info(),
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


def mlp_main(args, torch, svdq, synth):
    """fc1 (GELU) -> fc2 at M=4608: the fused step runs fc1's
    activation step, fc1's product whose epilogue writes fc2's codes, scales
    and h (svdq_w4a4_linear_requant), then fc2's product.  The unfused step
    stores fc1's Y and runs fc2's activation step on it."""
    prec = svdq.INT4 if args.prec == "int4" else svdq.MXFP4
    pre = "" if prec == svdq.INT4 else "mx_"
    f1s, f2s = synth.SPECS[pre + "fc1"], synth.SPECS[pre + "fc2"]
    g = svdq.group_of(prec)
    sdt = torch.float32 if prec == svdq.INT4 else torch.uint8
    M, K1, N1, N2, r = f1s.M, f1s.K, f1s.N, f2s.N, svdq.RANK
    print(f"[bench] generating and packing fc1 {M}x{K1}->{N1} and fc2 {M}x{N1}->{N2}", file=sys.stderr,
          flush=True)
    L1 = synth.make_layer(f1s)
    p1 = svdq.pack_weights(L1["W"], L1["act_absmax"], prec=prec)
    d1 = svdq.to_device(p1)
    b1 = svdq.bf16_tensor(L1["bias"])
    # fc2's calibration statistic comes from fc1's actual output
    X1 = svdq.bf16_tensor(L1["X"])
    xq, xs, h = svdq.quantize_act(X1, d1["smooth"], d1["down"], prec)
    Y1 = svdq.w4a4_linear(xq, xs, h, d1["wq"], d1["wscale"], d1["up"], b1, prec, svdq.EPI_GELU_TANH)
    L2 = synth.make_layer(f2s, X_bits=svdq.bf16_bits(Y1))
    p2 = svdq.pack_weights(L2["W"], L2["act_absmax"], prec=prec)
    del Y1, xq, xs, h
    sets = []
    for i in range(args.sets or 3):
        a, b = svdq.to_device(p1), svdq.to_device(p2)
        sets.append(dict(
            X=svdq.bf16_tensor(L1["X"]), d1=a, b1=svdq.bf16_tensor(L1["bias"]), d2=b,
            b2=svdq.bf16_tensor(L2["bias"]),
            xq=torch.empty((M, K1 // 2), dtype=torch.uint8, device="cuda"),
            xs=torch.empty((M, K1 // g), dtype=sdt, device="cuda"),
            h=torch.empty((M, r), dtype=torch.float32, device="cuda"),
            Y1=torch.empty((M, N1), dtype=torch.bfloat16, device="cuda"),
            xq2=torch.empty((M, N1 // 2), dtype=torch.uint8, device="cuda"),
            xs2=torch.empty((M, N1 // g), dtype=sdt, device="cuda"),
            h2=torch.empty((M, r), dtype=torch.float32, device="cuda"),
            work=torch.empty((svdq.requant_workspace_bytes(M, N1, prec=prec),), dtype=torch.uint8, device="cuda"),
            Y2=torch.empty((M, N2), dtype=torch.bfloat16, device="cuda")))

    def act1(b):
        svdq.quantize_act(b["X"], b["d1"]["smooth"], b["d1"]["down"], prec, xq=b["xq"], xscale=b["xs"], h=b["h"])

    def fc1_fused(b):
        d = b["d1"]
        svdq.w4a4_linear_requant(b["xq"], b["xs"], b["h"], d["wq"], d["wscale"], d["up"], b["b1"],
                                 b["d2"]["smooth"], b["d2"]["down"], prec, svdq.EPI_GELU_TANH,
                                 out=(b["xq2"], b["xs2"], b["h2"]), work=b["work"])

    def fc1_plain(b):
        d = b["d1"]
        svdq.w4a4_linear(b["xq"], b["xs"], b["h"], d["wq"], d["wscale"], d["up"], b["b1"], prec,
                         svdq.EPI_GELU_TANH, Y=b["Y1"])

    def act2(b):
        svdq.quantize_act(b["Y1"], b["d2"]["smooth"], b["d2"]["down"], prec, xq=b["xq2"], xscale=b["xs2"],
                          h=b["h2"])

    def fc2(b):
        d = b["d2"]
        svdq.w4a4_linear(b["xq2"], b["xs2"], b["h2"], d["wq"], d["wscale"], d["up"], b["b2"], prec,
                         svdq.EPI_NONE, Y=b["Y2"])

    fused = [act1, fc1_fused, fc2]
    plain = [act1, fc1_plain, act2, fc2]

    def run(seq, n, per_launch=False):
        evs = []
        for i in range(n):
            b = sets[i % len(sets)]
            if per_launch:
                e = [torch.cuda.Event(enable_timing=True) for _ in range(len(seq) + 1)]
                e[0].record()
                for j, f in enumerate(seq):
                    f(b)
                    e[j + 1].record()
                evs.append(e)
            else:
                for f in seq:
                    f(b)
        return evs

    for seq in (fused, plain):
        run(seq, args.warmup)
    torch.cuda.synchronize()
    print(f"[bench] warmup done; timing {args.steps} fused and {args.steps} unfused steps", file=sys.stderr,
          flush=True)
    out = {}
    # two rounds, fused and unfused alternating; the second round is reported
    # (the first one lets the clocks settle for both)
    for name, seq in (("fused", fused), ("plain", plain), ("fused", fused), ("plain", plain)):
        s0, s1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        s0.record()
        run(seq, args.steps)
        s1.record()
        torch.cuda.synchronize()
        out[name] = s0.elapsed_time(s1) / args.steps
        evs = run(seq, args.steps, per_launch=True)
        torch.cuda.synchronize()
        out[name + "_launch_ms"] = [round(float(np.mean([e[j].elapsed_time(e[j + 1]) for e in evs])), 5)
                                    for j in range(len(seq))]
    clock = gpu_clock(torch, lambda i: [f(sets[i % len(sets)]) for f in fused], out["fused"])
    ops = 2.0 * M * N1 * K1 + 2.0 * M * N2 * N1
    cpu = None
    if not args.no_cpu_baseline:
        from oracle import oracle as O
        print("[bench] timing the CPU oracle on a row sample of the pair", file=sys.stderr, flush=True)

        def oracle_rows(n):
            # fc1's activation step and product, its fp64 output rounded to
            # bf16 as fc2's input, fc2's activation step and product
            q, s_, hh = O.quant_act(L1["X"][:n], p1["smooth"], p1["down"], prec)
            y1 = O.linear(q, s_, hh, p1["wq"], p1["wscale"], p1["up"], L1["bias"], prec, gelu=True)
            q, s_, hh = O.quant_act(synth.f64_to_bf16_bits(y1), p2["smooth"], p2["down"], prec)
            O.linear(q, s_, hh, p2["wq"], p2["wscale"], p2["up"], L2["bias"], prec)

        rows = min(M, 32)
        t0 = time.time()
        oracle_rows(rows)
        probe = max(time.time() - t0, 1e-3)
        rows = int(min(M, max(8, rows * args.cpu_seconds / probe)))
        t0 = time.time()
        oracle_rows(rows)
        t_cpu = time.time() - t0
        cpu = {"value": round(ops * rows / M / t_cpu / 1e12, 6), "unit": "TOPS", "cores": O.num_threads(),
               "kind": "oracle",
               "sample": f"{rows} of {M} token rows through both layers (activation steps + products), "
                         f"{t_cpu:.1f} s"}
    req_ms = out["fused_launch_ms"][1]
    req_tops = 2.0 * M * N1 * K1 / (req_ms * 1e-3) / 1e12
    peak = PEAK_INT8_TOPS if prec == svdq.INT4 else PEAK_FP4_TFLOPS
    fmt = "INT4 g64" if prec == svdq.INT4 else "MXFP4 g32"
    line = {
        "metric": "fc1 -> fc2 MLP pair, fc2's activation step fused into fc1's epilogue (TOPS)",
        "value": round(ops / (out["fused"] * 1e-3) / 1e12, 2),
        "unit": "TOPS",
        "n_gpus": 1,
        "steps": args.steps,
        "warmup": args.warmup,
        "ms_per_step": round(out["fused"], 5),
        "higher_is_better": True,
        "scaling": "weak",
        "vs_baseline": None,
        "dtype": "int4 codes as exact fp8 E4M3 subnormals on the fp8 matrix cores (exact per-group partials); "
                 "group scale sx*sw from a bf16 hi/lo matrix product (~2^-16 relative), one fp32 fma per group"
                 if prec == svdq.INT4
                 else "mxfp4 (e2m1 x e2m1, e8m0 scales) on the scaled fp4 matrix cores, fp32 accumulation",
        "data": "synthetic (seeded Student-t activations with outlier channels, N(0,0.02^2) weights); "
                "fc2's input is fc1's GPU output",
        "config": {"workload": f"MLP: {M} tokens x {K1} -> {N1} (GELU) -> {N2}, rank {r}, {fmt}, bias; "
                               "fused step = quantize_act + w4a4_linear_requant + w4a4_linear; "
                               "unfused step = quantize_act + w4a4_linear + quantize_act + w4a4_linear",
                   "M": M, "K": K1, "N": N1, "N2": N2, "rank": r, "buffer_sets": len(sets)},
        "unfused_ms_per_step": round(out["plain"], 5),
        "fused_launch_ms": out["fused_launch_ms"],
        "unfused_launch_ms": out["plain_launch_ms"],
        "roofline": {"bound": "mfma", "kernel": "svdq_w4a4_linear_requant (fc1, with the h2 sum)",
                     "achieved": round(req_tops, 2), "peak": peak, "unit": "TFLOP/s",
                     "frac": round(req_tops / peak, 4), "traffic": None, "avg_ms": req_ms},
        "gpu_clock": clock,
        "host": host_info(),
        "cpu_baseline": cpu,
    }
    print(json.dumps(line), flush=True)


if __name__ == "__main__":
    main()
