"""The 8-bit floating-point layers in fp64 (torch), with elementwise error bounds for the kernels.

Error model, u = half a step of a type relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24):
  * products: the codes' products are exact in fp32 (2 x 4 significant bits).  A sum over L of them
    in fp32 is off by at most L 2^-23 S, S = sum |a||b| (two half steps per term, for the split of
    the sum over tensor-core steps and parts); the two scales and their use add 2^-22 S.
  * norm: a thread sums up to 32 squares, then there is a tree of at most 10 levels: rstd is off
    by (42 / 2) 2^-24 and a few roundings more, below 2^-18 in all; y by less than 2^-17.
  * activations: values within 2^-15 of themselves, derivatives within 2^-20 (absolute; see
    fused_ref).
  * a code is the nearest e4m3 number to v / scale, off by half its step.
"""
import math

import torch

from tests import fused_ref

BLOCK, TOP, FLOOR = 128, 448.0, 2.0 ** -100
F8 = torch.float8_e4m3fn
HALF = {torch.float16: (2.0 ** -11, 2.0 ** -25), torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}


def blocks(n):
    return -(-n // BLOCK)


def spread(scales, cols):
    """Scales [..., blocks] for each of the columns."""
    return scales.double().repeat_interleave(BLOCK, -1)[..., :cols]


def spread2(scales, rows, cols):
    return spread(scales, cols).repeat_interleave(BLOCK, -2)[..., :rows, :]


def tops(v):
    """max|v| of each block of the rows, NaN included."""
    pad = torch.nn.functional.pad(v, (0, -v.shape[-1] % BLOCK))
    return pad.unflatten(-1, (-1, BLOCK)).abs().amax(-1)


def quantize(v):
    """(codes, scales) of fp64 rows."""
    scales = (tops(v).clamp_min(FLOOR) / TOP).float()
    q = (v / spread(scales, v.shape[-1])).clamp(-TOP, TOP)
    return q.float().to(F8), scales


def weights(gen, *shape, device="cuda"):
    """Random codes (every finite one) and scales [..., N / 128, K / 128]."""
    codes = torch.randint(0, 256, shape, generator=gen, device=device, dtype=torch.int32)
    codes = torch.where(codes & 127 == 127, codes - 1, codes).to(torch.uint8).view(F8)
    scales = torch.rand(*shape[:-2], blocks(shape[-2]), blocks(shape[-1]), generator=gen,
                        device=device) * 1e-3 + 1e-5
    return codes, scales


def half_step(v):
    """Half a step of e4m3 at v (|v| <= 448)."""
    e = torch.frexp(v.abs())[1] - 1
    return torch.exp2((e.clamp_min(-6) - 4).double())


def check_codes(q, scales, v, err=0.0, what=""):
    """q, scales against fp64 values v that the kernel has to within err (a tensor or 0)."""
    assert q.dtype is F8 and scales.dtype is torch.float32
    err = err * torch.ones_like(v)
    s = (tops(v).clamp_min(FLOOR) / TOP)
    serr = tops(err) / TOP + 2.0 ** -23 * s
    assert scales.shape == s.shape
    off = (scales.double() - s).abs()
    assert bool((off <= serr).all()), f"{what} scales: {(off / serr).max().item():.3g} of the bound"
    full = spread(scales, v.shape[-1])
    x = v / full
    off = (q.double() - x.clamp(-TOP, TOP)).abs()
    bound = half_step(x.clamp(-TOP, TOP)) + err / full + x.abs() * 2.0 ** -22
    assert bool((off <= bound).all()), f"{what} codes: {(off / bound).max().item():.3g} of the bound"


def check(got, want, err, what=""):
    """A 16-bit output against fp64 values that the kernel has to within err before rounding."""
    u, tiny = HALF[got.dtype]
    bound = err * (1 + u) + u * want.abs() + tiny
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), f"{what}: {(off / bound).max().item():.3g} of the bound"


def product(q, scales, codes, wscales, backward=False):
    """(y, bound before rounding) in fp64."""
    N, K = codes.shape
    w = codes.double() * spread2(wscales, N, K)
    x = q.double() * spread(scales, q.shape[1])
    if not backward:
        w = w.t()
    return x @ w, (x.abs() @ w.abs()) * (q.shape[1] * 2.0 ** -23 + 2.0 ** -22)


def grouped(q, scales, offsets, codes, wscales, backward=False):
    """(first row, last row, y, bound) of the experts that have rows."""
    at = offsets.tolist()
    for e in range(codes.shape[0]):
        a, b = at[e], at[e + 1]
        if b > a:
            yield a, b, *product(q[a:b], scales[a:b], codes[e], wscales[e], backward)


def norm(x, residual, weight, eps):
    """(t as stored, rstd, y)."""
    t = x
    if residual is not None:
        t = (x.double() + residual.double()).to(x.dtype)
    v = t.double()
    rstd = (v.square().mean(1) + eps).rsqrt()
    return t, rstd, v * rstd[:, None] * weight.double()


def norm_backward(dy, total, rstd, weight, dtotal=None):
    """(dx, its bound, dweight, its bound)."""
    d, v, r, w = dy.double(), total.double(), rstd.double()[:, None], weight.double()
    n = v * r
    mean, mean_abs = (d * w * n).mean(1, keepdim=True), (d * w * n).abs().mean(1, keepdim=True)
    dx = r * (d * w - n * mean)
    err = r * ((d * w).abs() * 2.0 ** -21 + n.abs() * mean_abs * 2.0 ** -18)
    if dtotal is not None:
        dx = dx + dtotal.double()
        err = err + dx.abs() * 2.0 ** -24
    terms = d * n
    return dx, err, terms.sum(0), terms.abs().sum(0) * (dy.shape[0] + 8) * 2.0 ** -24 + 1e-42


def gated(gu, act):
    """(h, bound)."""
    g, u = gu.double().chunk(2, 1)
    h = fused_ref.act(act, g) * u
    return h, h.abs() * 2.0 ** -15 + 1e-37


def gated_backward(dh, gu, act):
    """((dg, du), bound)."""
    d = dh.double()
    g, u = gu.double().chunk(2, 1)
    f, df = fused_ref.act(act, g), fused_ref.act_grad(act, g)
    v = torch.cat([d * u * df, d * f], 1)
    err = torch.cat([(d * u).abs() * 2.0 ** -20, (d * f).abs() * 2.0 ** -15], 1)
    return v, err + v.abs() * 2.0 ** -21 + 1e-37


def activations(gen, M, K, dtype, std=1.0):
    x = torch.randn(M, K, generator=gen, device="cuda") * std
    return (x * torch.exp(0.5 * torch.randn(K, generator=gen, device="cuda"))).to(dtype)


def split(rows, E, rng, empty=0.3):
    """Ascending offsets of `rows` rows over E experts, about `empty` of them without rows."""
    share = [0.0 if rng.random() < empty else rng.random() ** 2 for _ in range(E)]
    total = sum(share) or 1.0
    at, run = [0], 0.0
    for s in share:
        run += s
        at.append(int(math.floor(run / total * rows + 0.5)))
    at[-1] = rows if sum(share) else 0
    for i in range(1, E + 1):
        at[i] = min(max(at[i], at[i - 1]), rows)
    return at
