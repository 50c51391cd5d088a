"""The fused linear layers in fp64 (torch), from the oracle's weights, with elementwise error
bounds for the fp16 kernels.

Error model, u = 2^-11 (half a step of fp16 relative to the value), t = 2^-25 (half a step of
its subnormals), S = sum |a||w| over the contraction of length L:
  * the operands: each fp16 weight is off by u (relative) + t, the gradient dz likewise;
  * the sum: fp32 accumulation over L terms, at most L 2^-23 S (two half steps per term, for
    the split of the sum over tensor-core steps and blocks);
  * an output is rounded once: u |y| + t.
Activations: |act'| <= 1.13 for every supported one, and their fp32 evaluation is off by at
most 2^-20 (|z| + 1).  The fp32 evaluation of act' itself has an absolute error: it is a sum
such as sigma + z sigma (1 - sigma) whose terms are each at most 1.2 in size and off by a few
2^-24 of that, and cancel where act' crosses zero, so no bound relative to |act'| holds there;
2^-20 bounds it (sixteen half steps of a value of 1).  dz is then off by 2^-20 |dy| (gated:
times |u|, and 2^-20 |dh| (|g| + 1) for the activation itself) before its rounding.
"""
import math

import numpy as np
import torch

import oracle

U, TINY, LIP = 2.0 ** -11, 2.0 ** -25, 1.13


def weight(layer, fmt):
    """fp64 [K, N] on the host."""
    if fmt == "lut4":
        return oracle.dequant_lut4(oracle.unpack_lut4(layer.qbytes), layer.lut, layer.absmax, 64)
    return oracle.dequant_uniform(oracle.unpack_uniform(layer.qweight, int(fmt[1:])),
                                  layer.scales, layer.zeros, 128)


def canonical(layer, fmt):
    if fmt == "lut4":
        return layer.qbytes, layer.lut, layer.absmax
    return layer.qweight, layer.scales, layer.zeros


def act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.relu(z)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z)


def act_grad(name, z):
    zz = z.detach().clone().requires_grad_(True)
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    return torch.autograd.grad(act(name, zz).sum(), zz)[0]


def product(a, w):
    """(a w, bound of the kernel's error before the output's rounding)."""
    s = a.abs() @ w.abs()
    return a @ w, s * (U + w.shape[0] * 2.0 ** -23) + TINY * a.abs().sum(1, keepdim=True)


def product_t(d, w, scale):
    """(d w^T, bound), d the unrounded gradient (rounded to fp16 by the kernel as well), off by
    2^-20 scale before that."""
    s = d.abs() @ w.abs().t()
    err = 2.0 ** -20 * scale @ w.abs().t() + s * (2.01 * U + w.shape[1] * 2.0 ** -23) + TINY * d.abs().sum(1, keepdim=True)
    return d @ w.t(), err + TINY * w.abs().sum(1)


def rounded(y, err):
    return err * (1 + U) + U * y.abs() + TINY


def linear(x, w, bias=None, residual=None, name="none"):
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias
        ez = ez + 2.0 ** -23 * z.abs()
    y = act(name, z)
    ey = LIP * ez + 2.0 ** -20 * (z.abs() + 1) * (name != "none")
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -23 * y.abs()
    return (y, rounded(y, ey)), (z, rounded(z, ez))


def gated(x, wg, wu, bias=None, name="silu"):
    (g, eg), (u, eu) = product(x, wg), product(x, wu)
    if bias is not None:
        g, u = g + bias[0], u + bias[1]
        eg, eu = eg + 2.0 ** -23 * g.abs(), eu + 2.0 ** -23 * u.abs()
    a = act(name, g)
    ea = LIP * eg + 2.0 ** -20 * (g.abs() + 1)
    h = a * u
    eh = ea * u.abs() + a.abs() * eu + ea * eu
    gu, egu = torch.stack([g, u], 1), torch.stack([eg, eu], 1)
    return (h, rounded(h, eh)), (gu, rounded(gu, egu))


def column_sums(dz, scale):
    """(sum over rows, bound): fp32 sums of elements off by 2^-20 scale."""
    s = dz.abs().sum(0)
    return dz.sum(0), s * dz.shape[0] * 2.0 ** -24 + 2.0 ** -20 * scale.sum(0) + 2.0 ** -40


def linear_backward(dy, z, w, name):
    dz = dy * act_grad(name, z) if name != "none" else dy
    scale = dy.abs() * (name != "none")
    dx, e = product_t(dz, w, scale)
    return (dx, rounded(dx, e)), column_sums(dz, scale)


def gated_backward(dh, gu, wg, wu, name):
    g, u = gu[:, 0], gu[:, 1]
    dg, du = dh * u * act_grad(name, g), dh * act(name, g)
    scale = torch.stack([(dh * u).abs(), dh.abs() * (g.abs() + 1)], 1)
    dx, e = product_t(torch.cat([dg, du], 1), torch.cat([wg, wu], 1), scale.flatten(1))
    return (dx, rounded(dx, e)), column_sums(torch.stack([dg, du], 1), scale)


# Relative L2: each output carries at most three roundings (weight or gradient operands, the
# output) of rms at most u / sqrt(3) of the value each, 4.9e-4 together, a gated product two
# more; twice that is allowed.
REL = 1.3e-3


def check(got, want, what=""):
    ref, bound = want
    got = got.double()
    assert got.shape == ref.shape, what
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outputs beyond the "
                           f"bound, worst {float((err / bound).max()):.2f} of it")
    norm = float(ref.norm())
    if norm > 0 and got.numel() >= 256:
        assert float(err.norm()) <= REL * norm, f"{what}: relL2 {float(err.norm()) / norm:.2e}"


def seeded(seed, *shape, std=1.0):
    """fp16 normal values as a numpy array."""
    r = np.random.default_rng([seed, 77])
    return (r.standard_normal(shape) * std).astype(np.float16)
