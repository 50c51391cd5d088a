"""Time the 8-bit floating-point layers of one shape: RMS norm, gated activation and quantization
with e4m3 output, and the products, dense or grouped by expert, with their backward passes.

    python -m weight_only_quantized_gemv_b200.run_fp8 --K 8192 --N 28672 --M 512 [--E 8] \
        [--only linear|norm|...] [--type bfloat16] [--act silu] [--time]

K: columns of the norm and of the product's input; N: columns of the product's output and 2 F of the
gated activation.  With --E the product's rows are spread over that many matrices, some with twice
the average and some with none.  Enough copies of the weights are cycled that no launch finds them
in L2 (the row kernels' inputs may be there).  Without `--time` the chosen entries run `--launches`
times (for profiler captures); with it each is timed with CUDA events on the launching stream after
warm-up, and one JSON line gives microseconds, GB/s (every input read once, every output written
once) and for products TFLOP/s.
"""
from __future__ import annotations

import argparse
import json
import math

import torch

from . import ACTS, TYPES
from .layers import (Fp8Experts, Fp8Linear, RMSNorm, fp8_gated, fp8_gated_backward, fp8_quantize,
                     fp8_quantize_weights)

L2_BYTES = 126 * 2 ** 20
ENTRIES = ("quantize", "norm", "norm_backward", "gated", "gated_backward", "linear",
           "linear_backward")


def moved_bytes(entry: str, M: int, N: int, K: int, matrices: int = 1) -> int:
    """Bytes an entry cannot do without; 16-bit values, codes and their scales."""
    def coded(columns):
        return M * columns + 4 * M * -(-columns // 128)

    if entry == "quantize":
        return 2 * M * K + coded(K)
    if entry == "norm":       # x, residual, total
        return 6 * M * K + 2 * K + coded(K)
    if entry == "norm_backward":  # dy, total, dtotal, dx
        return 8 * M * K + 4 * M + 6 * K
    if entry == "gated":
        return 2 * M * N + coded(N // 2)
    if entry == "gated_backward":
        return 3 * M * N + coded(N)
    weights = matrices * (N * K + 4 * -(-N // 128) * -(-K // 128))
    inner, outer = (N, K) if entry.endswith("backward") else (K, N)
    return weights + coded(inner) + 2 * M * outer


def ragged_offsets(M: int, E: int) -> list:
    """Row ranges of E experts: every fourth has none, the others share M rows unevenly."""
    share = [0 if e % 4 == 3 and E > 1 else 1 + e % 3 for e in range(E)]
    at, run = [0], 0
    for s in share:
        run += s
        at.append(M * run // sum(share))
    return at


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--K", type=int, default=8192)
    ap.add_argument("--N", type=int, default=28672)
    ap.add_argument("--M", type=int, default=512)
    ap.add_argument("--E", type=int, default=0)
    ap.add_argument("--type", choices=sorted(TYPES), default="bfloat16")
    ap.add_argument("--act", choices=sorted(ACTS), default="silu")
    ap.add_argument("--only", choices=ENTRIES, default=None)
    ap.add_argument("--launches", type=int, default=4)
    ap.add_argument("--reps", type=int, default=20)
    ap.add_argument("--time", action="store_true")
    a = ap.parse_args()
    K, N, M, E, dtype = a.K, a.N, a.M, a.E, getattr(torch, a.type)
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    gen = torch.Generator(device=dev).manual_seed(0)

    def values(*shape, std=1.0):
        return (torch.randn(*shape, device=dev, generator=gen) * std).to(dtype)

    lead = (E,) if E else ()
    copies = max(2, math.ceil(2 * L2_BYTES / (max(E, 1) * N * K)))
    kind = Fp8Experts if E else Fp8Linear
    mats = [kind(*fp8_quantize_weights(values(*lead, N, K, std=0.02))) for _ in range(copies)]
    at = ragged_offsets(M, E) if E else None
    rows = (torch.tensor(at, dtype=torch.int32, device=dev),) if E else ()
    matrices = sum(b > a_ for a_, b in zip(at, at[1:])) if E else 1

    x, r, dy, gu, dh = values(M, K), values(M, K), values(M, K), values(M, N), values(M, N // 2)
    norm, total, rstd = RMSNorm(values(K)), torch.empty_like(x), torch.empty(M, device=dev)
    dweight = torch.empty(K, device=dev)
    qx, qd = fp8_quantize(x), fp8_quantize(gu)
    norm.forward(x, r, total=total, rstd=rstd)
    for lay in mats:
        lay.reserve(M)

    def run(entry, i):
        if entry == "quantize":
            fp8_quantize(x)
        elif entry == "norm":
            norm.forward(x, r, total=total)
        elif entry == "norm_backward":
            norm.backward(dy, x, rstd, dtotal=r, dweight=dweight)
        elif entry == "gated":
            fp8_gated(gu, a.act)
        elif entry == "gated_backward":
            fp8_gated_backward(dh, gu, a.act)
        elif entry == "linear":
            mats[i % copies].forward(*qx, *rows, dtype=dtype)
        else:
            mats[i % copies].backward(*qd, *rows, dtype=dtype)

    out = {"K": K, "N": N, "M": M, "E": E, "type": a.type, "act": a.act}
    for entry in [a.only] if a.only else ENTRIES:
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
        out[entry] = {"us": round(us, 2),
                      "GBs": round(moved_bytes(entry, M, N, K, matrices) / us / 1e3, 1)}
        if entry.startswith("linear"):
            out[entry]["TFLOPs"] = round(2 * M * N * K / us / 1e6, 1)
    torch.cuda.synchronize()
    out["error_flags"] = 0
    for lay in mats:
        out["error_flags"] |= lay.fused_read_error()
    print(json.dumps(out))


if __name__ == "__main__":
    main()
