"""The activations of the fused layers over every fp16 argument up to 16 in size, on the GPU,
against fp64: x = 0 and the argument as the bias, so that the pre-activation is exact and only the
activation's fp32 evaluation and the output's rounding are seen.

Bound of a value: half an fp16 step, u |y| (u = 2^-11) or 2^-25 below 2^-14, and EVAL |y| for the
evaluation.  EVAL: each value is a product z s (u) of a sigmoid or normal CDF s, whose relative
error is
  * that of its exponential, e^-a for |a| <= 30 (beyond it no output is larger than 2^-25):
    2 + 1.173 a ulp of 2^-23 (4.4e-6) and a's own rounding, five of 2^-24 for tanh-GELU's cubic
    (9e-6);
  * the division's 2 ulp, the polynomial's 1.5e-6 in fp32 and three products: 2e-6.
Together below 1.6e-5 < 2^-15.
"""
import functools
import math

import numpy as np
import pytest

from synth import gen
from tests import fused_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers

DEV = "cuda:0"
ACTS = ["relu", "gelu", "gelu_tanh", "silu"]
K = 128
EVAL = 2.0 ** -15


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@functools.lru_cache(maxsize=1)
def _arguments():
    """Every fp16 value from -16 to 16, filled up to a multiple of 16."""
    pos = np.arange(0, 0x4C00 + 1, dtype=np.uint16)
    z = np.concatenate([pos, pos | 0x8000]).view(np.float16)
    z = np.concatenate([z, z[:-len(z) % 16]])
    return torch.from_numpy(z).to(DEV)


@functools.lru_cache(maxsize=1)
def _layer():
    N = _arguments().numel()
    lay, up = (gen.uniform_layer(s, K, N, 4) for s in (1, 2))
    parts = [(u.qweight, u.scales, u.zeros) for u in (lay, up)]
    return (layers.QuantLinear(4, K, N, *parts[0], device=DEV),
            layers.GatedLinear(4, K, N, *parts, device=DEV))


def _value(name, z):
    """fp64, no cancellation in the tails."""
    if name == "relu":
        return z.clamp_min(0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z)


def _check(got, want, what):
    want = want.expand_as(got)
    bound = want.abs() * (ref.U + EVAL) + ref.TINY
    err = (got.double() - want).abs()
    worst = (err / bound).max()
    assert worst <= 1, f"{what}: {float(worst):.3f} of the bound"


@pytest.mark.parametrize("M", [1, 9, 20, 100])
@pytest.mark.parametrize("act", ACTS)
def test_values_in_the_tails(act, M):
    """The GEMV's epilogue (1 and 9 rows) and the product's (one CTA and a pair)."""
    z = _arguments()
    lay, _ = _layer()
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    kept = torch.empty((M, z.numel()), dtype=torch.float16, device=DEV)
    y = lay.linear(x, bias=z, act=act, z=kept)
    assert torch.equal(kept, z.expand_as(kept))
    _check(y, _value(act, z.double()), act)


@pytest.mark.parametrize("factor", [1.0, -1000.0, 30000.0])
@pytest.mark.parametrize("M", [1, 9, 20, 100])
@pytest.mark.parametrize("act", ACTS)
def test_gated_values_in_the_tails(act, M, factor):
    """A large up value shows the relative error of a small activation."""
    z = _arguments()
    _, gat = _layer()
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    bias = torch.stack([z, torch.full_like(z, factor)])
    h = gat.forward(x, bias=bias, act=act)
    want = _value(act, z.double()) * factor
    keep = want.abs() < 65504
    _check(h[:, keep], want[keep], f"{act} times {factor}")


def _derivative(name, z):
    """fp64: (act', the sum of the sizes of its terms, the sigmoid's argument or 0)."""
    zero = torch.zeros_like(z)
    if name == "relu":
        return (z > 0).double(), zero, zero
    if name == "gelu":
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        cdf = 0.5 * torch.erfc(-z * math.sqrt(0.5))
        return cdf + z * phi, cdf + (z * phi).abs(), zero
    a, slope = z, torch.ones_like(z)
    if name == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        a, slope = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(a)
    t = z * s * torch.sigmoid(-a) * slope
    return s + t, s + t.abs(), a.abs() if name == "gelu_tanh" else zero


@pytest.mark.parametrize("act", ACTS)
def test_gradients_in_the_tails(act):
    """The fp32 column sums of one row of ones are the derivatives themselves.  Relative to their
    terms: a sigmoid and its complement are each within 2 ulp of the exponential and three half
    steps more, 4.2e-7, a product of both and z within 2^-20; the tanh form's argument adds its
    own five half steps (2^-21.6 |a|); the normal CDF's polynomial is within 1.5e-6 (2^-19), the
    density's argument exact."""
    z = _arguments()
    lay, gat = _layer()
    N = z.numel()
    one = torch.ones((1, N), dtype=torch.float16, device=DEV)
    db = torch.empty(N, dtype=torch.float32, device=DEV)
    lay.linear_backward(one, z=z.view(1, N), act=act, dbias=db)
    want, terms, a = _derivative(act, z.double())
    rel = 2.0 ** -19 if act == "gelu" else 2.0 ** -20 * (1 + a)
    worst = ((db.double() - want).abs() / (rel * terms + 2.0 ** -126)).max()
    assert worst <= 1, f"{float(worst):.3f} of the bound"
    both = torch.empty((2, N), dtype=torch.float32, device=DEV)
    gat.backward(one, torch.stack([z, torch.ones_like(z)]).view(1, 2, N), act=act, dbias=both)
    assert torch.equal(both[0], db)
    value = _value(act, z.double())
    worst = ((both[1].double() - value).abs() / (rel * value.abs() + 2.0 ** -126)).max()
    assert worst <= 1, f"value: {float(worst):.3f} of the bound"
