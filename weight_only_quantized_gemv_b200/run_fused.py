"""Time the fused linear layers of one shape: the product with bias, activation and residual,
the gated projection, and the backward passes of both.

    python -m weight_only_quantized_gemv_b200.run_fused --fmt w4 --K 8192 --N 28672 --M 512 \
        [--only linear|gated|linear_backward|gated_backward] [--act silu] [--plain] [--time]

N: columns of the packed weights (gated: 2 F).  Packed codes and parameters are random bytes
of the right sizes; enough copies of them are cycled that no launch finds its weights in L2.
Without `--time` the chosen entries run `--launches` times (for profiler captures); with it
each is timed with CUDA events on the launching stream after warm-up, and one JSON line gives
microseconds, TFLOP/s (2 M N K) and GB/s (weights, activations and outputs once).  `--plain`
leaves out bias, residual, kept pre-activations and bias gradients.
"""
from __future__ import annotations

import argparse
import json
import math

import torch

from . import (ACTS, FORMATS, QL_FMT_LUT4, qlinear_fused_workspace_bytes, qlinear_gated,
               qlinear_gated_backward, qlinear_linear, qlinear_linear_backward,
               qlinear_read_error)

L2_BYTES = 126 * 2 ** 20
ENTRIES = ("linear", "gated", "linear_backward", "gated_backward")


def moved_bytes(entry: str, fmt: int, M: int, N: int, K: int, act: str, plain: bool) -> int:
    """Bytes an entry cannot do without: every input read once, every output written once."""
    weights = (K * N // 2 + (K // 64) * N * 4 + 32 if fmt == QL_FMT_LUT4
               else K * N * fmt // 8 + 4 * (K // 128) * N)
    width = N // 2 if entry.startswith("gated") else N
    if entry.endswith("backward"):
        kept = M * N if entry.startswith("gated") or act != "none" else 0
        return weights + 2 * (M * width + kept + M * K) + (0 if plain else 4 * N)
    extra = 0 if plain else 2 * N + 2 * M * N + (2 * M * N if entry == "linear" else 0)
    return weights + 2 * (M * K + M * width) + extra


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--fmt", choices=["w2", "w4", "w8", "lut4"], default="w4")
    ap.add_argument("--K", type=int, default=8192)
    ap.add_argument("--N", type=int, default=28672)
    ap.add_argument("--M", type=int, default=512)
    ap.add_argument("--act", choices=sorted(ACTS), default="silu")
    ap.add_argument("--only", choices=ENTRIES, default=None)
    ap.add_argument("--plain", action="store_true")
    ap.add_argument("--launches", type=int, default=4)
    ap.add_argument("--reps", type=int, default=20)
    ap.add_argument("--time", action="store_true")
    a = ap.parse_args()
    fmt, K, N, M = FORMATS[a.fmt], a.K, a.N, a.M
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    bits = 4 if fmt == QL_FMT_LUT4 else fmt
    per_copy = K * N * bits // 8
    copies = max(2, math.ceil(2 * L2_BYTES / per_copy))
    gen = torch.Generator(device=dev).manual_seed(0)
    q = [torch.randint(0, 256, (per_copy,), dtype=torch.uint8, device=dev, generator=gen)
         for _ in range(copies)]
    if fmt == QL_FMT_LUT4:
        p0 = torch.linspace(-1, 1, 16, device=dev).half()
        p1 = torch.rand((K // 64) * N, device=dev, generator=gen) * 0.05
    else:
        p0 = (torch.rand((K // 128) * N, device=dev, generator=gen) * 0.01).half()
        p1 = torch.randint(0, 1 << bits, ((K // 128) * N,), device=dev, generator=gen).half()

    def half(*shape):
        return torch.randn(*shape, device=dev, generator=gen).half()

    x, z, bias = half(M, K), half(M, N), half(N)
    d, dh, res = half(M, N), half(M, N // 2), half(M, N)
    y, h, dx = half(M, N), half(M, N // 2), half(M, K)
    kept, db = half(M, N), torch.empty(N, device=dev)
    if a.plain:
        bias = res = kept = db = None
    ws = torch.zeros(qlinear_fused_workspace_bytes(fmt, M, N, K), dtype=torch.uint8, device=dev)

    def run(entry, i):
        w = (q[i % copies], p0, p1)
        if entry == "linear":
            qlinear_linear(fmt, x, *w, y, M, N, K, ws, bias, res, a.act, kept)
        elif entry == "gated":
            qlinear_gated(fmt, x, *w, h, M, N // 2, K, ws, bias, a.act, kept)
        elif entry == "linear_backward":
            qlinear_linear_backward(fmt, d, z, *w, dx, M, N, K, ws, a.act, db)
        else:
            qlinear_gated_backward(fmt, dh, z, *w, dx, M, N // 2, K, ws, a.act, db)

    entries = [a.only] if a.only else list(ENTRIES)
    out = {"fmt": a.fmt, "K": K, "N": N, "M": M, "act": a.act, "plain": a.plain}
    for entry in entries:
        if not a.time:
            for i in range(a.launches):
                run(entry, i)
            continue
        for i in range(2 * copies):
            run(entry, i)
        torch.cuda.synchronize()
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record()
        for i in range(a.reps):
            run(entry, i)
        e1.record()
        torch.cuda.synchronize()
        us = e0.elapsed_time(e1) * 1e3 / a.reps
        out[entry] = {"us": round(us, 2), "TFLOPs": round(2 * M * N * K / us / 1e6, 1),
                      "GBs": round(moved_bytes(entry, fmt, M, N, K, a.act, a.plain) / us / 1e3, 1)}
    torch.cuda.synchronize()
    out["error_flags"] = qlinear_read_error(ws)
    print(json.dumps(out))


if __name__ == "__main__":
    main()
