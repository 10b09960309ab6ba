"""Times one library entry point on one shape and prints a JSON line.

    python -m fp8_block_scaled_sgq_gb300.measure PATH M N K [--blk B] [--format F] [--reps R]

PATH is one of
  quant_per_token   sgq_quant_per_token on x [M, K]            (GB/s: 2 B in + 1 B code per element + 4 B per row)
  quant_per_tensor  sgq_quant_per_tensor, dynamic, on x [M, K] (GB/s: 2 B in + 1 B code per element)
  quant_v2          sgq_quant_token_group_v2, fused SiLU-and-mul, x [1, M, 2K] -> [1, M, K], group --blk, UE8M0
                    (GB/s: 4 B in + 1 B code per output element + 4 B per group)
  scaled_mm         sgq_fp8_scaled_mm, per-row x per-column scales, bias   (TFLOP/s and GB/s)
  block_gemm        sgq_fp8_block_gemm with [B, B] blocks, UE8M0           (TFLOP/s and GB/s)
  linear            sgq_fp8_block_linear with [B, B] blocks, UE8M0         (GB/s of x + W + D)
  pair              sgq_quant_token_group then sgq_fp8_block_gemm, back to back on one stream
                    (programmatic dependent launch), [B, B] blocks, UE8M0  (TFLOP/s; GB/s of the
                    quantiser's and the GEMM's algorithmic bytes)
  quant_fp4         sgq_quant_fp4 on x [M, K], --format mxfp4 or nvfp4     (GB/s)
  dequant_fp4       sgq_dequant_fp4 to [M, K]                              (GB/s)
  fp4_gemm          sgq_fp4_gemm                                           (TFLOP/s and GB/s)
  norm              sgq_norm: norm of x [M, K], residual added, next norm into the format   (GB/s)

The metric's own configurations (the M = 1..8192 sweep, the prefill GEMMs and
the quantiser at prefill sizes) are timed by bench.py; this times the other
entry points, one shape at a time.

Timing: CUDA events around one replay of a CUDA graph holding `reps` calls on
one stream, after a warm-up replay; weights (and, for the quantisers, inputs)
rotate over enough copies to exceed twice the L2 size, so they come from HBM.
Inputs are seeded synthetic (x ~ N(0,1), W ~ N(0, 0.02)).
"""
from __future__ import annotations

import argparse
import json
import math

import torch

from . import binding, synth

L2_BYTES = 129 * 2 ** 20


FP4_PATHS = ["quant_fp4", "dequant_fp4", "fp4_gemm", "norm"]
PATHS = ["quant_per_token", "quant_per_tensor", "quant_v2", "scaled_mm", "block_gemm", "linear", "pair"] + FP4_PATHS


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("path", choices=PATHS)
    ap.add_argument("M", type=int)
    ap.add_argument("N", type=int)
    ap.add_argument("K", type=int)
    ap.add_argument("--blk", type=int, default=128)
    ap.add_argument("--format", choices=("mxfp4", "nvfp4"), default="nvfp4")
    ap.add_argument("--reps", type=int, default=50)
    args = ap.parse_args()
    print(json.dumps(measure(args.path, args.M, args.N, args.K, args.blk, args.reps, args.format)), flush=True)


def fp4_calls(path: str, M: int, N: int, K: int, fmt: str, dev):
    """The calls of a 4-bit path over rotating copies: (calls, bytes a call moves at least, operations)."""
    from . import dequant_fp4, fp4_gemm, norm_add, quant_fp4
    packed = lambda rows: rows * K // 2 + rows * K // (32 if fmt == "mxfp4" else 16)  # noqa: E731
    moved = {"quant_fp4": 2 * M * K + packed(M), "dequant_fp4": 2 * M * K + packed(M), "norm": 6 * M * K + packed(M),
             "fp4_gemm": packed(M) + packed(N) + 2 * M * N}[path]
    n_rot = max(2, math.ceil(2 * L2_BYTES / moved) + 1)
    calls = []
    if path == "fp4_gemm":
        xq, xs = quant_fp4(synth.activation(M, K, seed=1).to(dev), fmt)
        wq, ws = quant_fp4(synth.weight(N, K, seed=2).to(dev), fmt)
        d = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        rot = [(wq.clone(), ws.clone()) for _ in range(n_rot)]
        for w in rot:
            calls.append(lambda sp, w=w: fp4_gemm(xq, xs, *w, fmt, out=d, stream=sp))
        return calls, moved, 2 * M * N * K
    x = synth.activation(M, K, seed=1).to(dev)
    q, s = quant_fp4(x, fmt)
    y, one = torch.empty_like(x), torch.ones(K, dtype=x.dtype, device=dev)
    for _ in range(n_rot):
        if path == "quant_fp4":
            calls.append(lambda sp, x=x.clone(): quant_fp4(x, fmt, xq=q, xs=s, stream=sp))
        elif path == "dequant_fp4":
            calls.append(lambda sp, q=q.clone(), s=s.clone(): dequant_fp4(q, s, fmt, out=y, stream=sp))
        else:
            calls.append(lambda sp, x=x.clone(), r=x.clone(): norm_add(x, r, post_weight=one, weight=one, quant=fmt, h_out=y,
                                                                       out=q, out_scales=s, stream=sp))
    return calls, moved, 0


def measure(path: str, M: int, N: int, K: int, blk: int, reps: int, fmt: str = "nvfp4") -> dict:
    args = argparse.Namespace(path=path, reps=reps)
    dev = torch.device("cuda:0")
    st = torch.cuda.Stream()
    s = st.cuda_stream
    quant = args.path.startswith("quant") or path in FP4_PATHS
    rot_bytes = (M * K * (4 if args.path == "quant_v2" else 2)) if quant else N * K
    n_rot = max(2, math.ceil(2 * L2_BYTES / rot_bytes) + 1)
    calls = []
    if path in FP4_PATHS:
        calls, moved, flops = fp4_calls(path, M, N, K, fmt, dev)
        n_rot = len(calls)
        torch.cuda.synchronize()
    elif quant:
        W = 2 * K if args.path == "quant_v2" else K
        xr = [synth.activation(M, W, seed=i).to(dev) for i in range(min(n_rot, 4))]
        xr = [xr[i % len(xr)].clone() for i in range(n_rot)]
        xq = torch.empty((M, K), dtype=torch.uint8, device=dev)
        sc = torch.empty((max(M, 4),), dtype=torch.float32, device=dev)
        sc2 = torch.empty((M, K // blk), dtype=torch.float32, device=dev)
        for r in range(n_rot):
            if args.path == "quant_per_token":
                calls.append(lambda sp, r=r: binding.sgq_quant_per_token(xr[r], M, K, xq, sc, sp))
            elif args.path == "quant_v2":
                calls.append(lambda sp, r=r: binding.sgq_quant_token_group_v2(xr[r], 1, M, K, blk, 1, 1, None, xq,
                                                                             sc2, sp))
            else:
                calls.append(lambda sp, r=r: binding.sgq_quant_per_tensor(xr[r], M * K, 0, xq, sc, sp))
        moved = {"quant_per_token": M * K * 3 + 4 * M, "quant_per_tensor": M * K * 3 + 4,
                 "quant_v2": M * K * 5 + 4 * M * (K // blk)}[args.path]
        flops = 0
    else:
        x = synth.activation(M, K, seed=1).to(dev)
        w = synth.weight(N, K, seed=2).to(dev)
        d = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if args.path == "scaled_mm":
            wq0 = torch.empty((N, K), dtype=torch.uint8, device=dev)
            sb0 = torch.empty((N,), dtype=torch.float32, device=dev)
            binding.sgq_quant_per_token(w, N, K, wq0, sb0, s)
            aq = torch.empty((M, K), dtype=torch.uint8, device=dev)
            sa = torch.empty((M,), dtype=torch.float32, device=dev)
            binding.sgq_quant_per_token(x, M, K, aq, sa, s)
            bias = synth.activation(1, N, seed=3).reshape(N).to(dev)
            wrot = [(wq0, sb0)] + [(wq0.clone(), sb0.clone()) for _ in range(n_rot - 1)]
            for r in range(n_rot):
                calls.append(lambda sp, r=r: binding.sgq_fp8_scaled_mm(aq, sa, M, wrot[r][0], wrot[r][1], N, bias, d,
                                                                      M, N, K, sp))
            moved = M * K + 4 * M + N * K + 4 * N + 2 * N + 2 * M * N
        else:
            nb, kb = -(-N // blk), K // blk
            wq0 = torch.empty((N, K), dtype=torch.uint8, device=dev)
            ws0 = torch.empty((nb, kb), dtype=torch.float32, device=dev)
            binding.sgq_quant_weight_block(w, N, K, blk, blk, 1, wq0, ws0, s)
            wrot = [(wq0, ws0)] + [(wq0.clone(), ws0.clone()) for _ in range(n_rot - 1)]
            if args.path == "block_gemm":
                aq = torch.empty((M, K), dtype=torch.uint8, device=dev)
                as_ = torch.empty((M, K // blk), dtype=torch.float32, device=dev)
                binding.sgq_quant_token_group(x, M, K, blk, 1, aq, as_, s)
                for r in range(n_rot):
                    calls.append(lambda sp, r=r: binding.sgq_fp8_block_gemm(aq, as_, wrot[r][0], wrot[r][1], d, M, N,
                                                                           K, blk, blk, sp))
                moved = M * K + 4 * M * (K // blk) + N * K + 4 * nb * kb + 2 * M * N
            elif args.path == "pair":
                aq = torch.empty((M, K), dtype=torch.uint8, device=dev)
                as_ = torch.empty((M, K // blk), dtype=torch.float32, device=dev)

                def pair_call(sp, r):
                    binding.sgq_quant_token_group(x, M, K, blk, 1, aq, as_, sp)
                    binding.sgq_fp8_block_gemm(aq, as_, wrot[r][0], wrot[r][1], d, M, N, K, blk, blk, sp)
                for r in range(n_rot):
                    calls.append(lambda sp, r=r: pair_call(sp, r))
                moved = (2 * M * K + M * K + 4 * M * (K // blk)) + (M * K + 4 * M * (K // blk) + N * K
                                                                    + 4 * nb * kb + 2 * M * N)
            else:
                for r in range(n_rot):
                    calls.append(lambda sp, r=r: binding.sgq_fp8_block_linear(x, 1, wrot[r][0], wrot[r][1], d, M, N,
                                                                             K, blk, blk, None, None, sp))
                moved = 2 * M * K + N * K + 4 * nb * kb + 2 * M * N
        flops = 2 * M * N * K
    st.synchronize()
    with torch.cuda.stream(st):
        for i in range(n_rot):
            calls[i](s)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            sp = torch.cuda.current_stream().cuda_stream
            for i in range(args.reps):
                calls[i % n_rot](sp)
    with torch.cuda.stream(st):
        g.replay()
    st.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(st):
        e0.record(st)
        g.replay()
        e1.record(st)
    st.synchronize()
    us = e0.elapsed_time(e1) * 1e3 / args.reps
    status = binding.sgq_device_status(s)
    if status != 0:
        raise RuntimeError(f"device status {binding.status_string(status)}")
    out = {"path": args.path, "M": M, "N": N, "K": K, "us": round(us, 3), "gbs": round(moved / us / 1e3, 1)}
    if path in FP4_PATHS:
        out["format"] = fmt
    if flops:
        out["tflops"] = round(flops / us / 1e6, 2)
        out["blk"] = blk if args.path in ("block_gemm", "linear", "pair") else None
    del calls, g
    torch.cuda.empty_cache()
    return out


if __name__ == "__main__":
    main()
