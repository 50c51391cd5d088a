"""Backward passes of the fused layers whose gradients leave fp16's range before the product, on the
GPU, against fp64.

The kernels round dz to fp16 after scaling its row so that its largest |dy| (gated: |dh u|, |dh g|),
`top`, lies in [2^14, 2^15).  Bound of an output before its own rounding, S = sum |dz||w| over the
N columns:
  * operands: u S for the weights, u S for dz (u = 2^-11; both with their product: 2.01 u);
    2^-25 sum |dz| for subnormal weights; 2^-25 / 2^14 of the row's top for dz elements below
    the scaled row's normal range, times sum |w|;
  * the fp32 evaluation of dz: 2^-20 of dy (gated: dh u, dh (|g| + 1));
  * the sum: N 2^-23 S.
"""
import functools

import pytest

from synth import gen
from tests import fused_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@functools.lru_cache(maxsize=8)
def _layer(K, N, seed, power):
    """W4 with weights of 0.02 times 2^power."""
    u = gen.uniform_layer(seed, K, N, 4)
    u.scales = (u.scales.astype("float32") * 2.0 ** power).astype("float16")
    return u, torch.from_numpy(ref.weight(u, "w4")).to(DEV)


def _linear(K, N, power):
    u, w = _layer(K, N, 80, power)
    return layers.from_uniform(u, DEV), w


def _gated(K, F, power):
    (a, wa), (b, wb) = _layer(K, F, 81, power), _layer(K, F, 82, power)
    parts = [(u.qweight, u.scales, u.zeros) for u in (a, b)]
    return layers.GatedLinear(ql.QL_FMT_W4, K, F, *parts, device=DEV), wa, wb


def _t(seed, *shape, std=1.0):
    return torch.from_numpy(ref.seeded(seed, *shape, std=std)).to(DEV)


def _check(dx, d, scale, top, w):
    want = d @ w.t()
    s = d.abs() @ w.abs().t()
    err = s * (2.01 * ref.U + w.shape[1] * 2.0 ** -23) + ref.TINY * d.abs().sum(1, keepdim=True)
    err = err + 2.0 ** -39 * top.amax(1, keepdim=True) * w.abs().sum(1)
    err = err + 2.0 ** -20 * scale @ w.abs().t()
    bound = ref.rounded(want, err)
    off = (dx.double() - want).abs()
    assert bool((off <= bound).all()), f"worst {float((off / bound).max()):.2f} of the bound"
    # in the relative L2 norm (fused_ref.REL), and outputs below 2^-14 are rounded by up to 2^-25
    # whatever their size: at most 2^-25 sqrt(count) together
    assert float(off.norm()) <= ref.REL * float(want.norm()) + ref.TINY * off.numel() ** 0.5


def _linear_case(lay, w, dy, z, act):
    d = dy.double() * ref.act_grad(act, z.double())
    _check(lay.linear_backward(dy, z=z, act=act), d, dy.double().abs(), dy.double().abs(), w)


def _gated_case(lay, wg, wu, dh, gu, act):
    g, u, h = gu[:, 0].double(), gu[:, 1].double(), dh.double()
    d = torch.cat([h * u * ref.act_grad(act, g), h * ref.act(act, g)], 1)
    scale = torch.cat([(h * u).abs(), h.abs() * (g.abs() + 1)], 1)
    dx = lay.backward(dh, gu, act=act)
    assert torch.isfinite(dx).all()
    top = torch.cat([(h * u).abs(), (h * g).abs()], 1)
    _check(dx, d, scale, top, torch.cat([wg, wu], 1))


SHAPES = [(256, 208), (256, 2048), (128, 18944)]  # the last: rows wider than a block keeps


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [1, 17, 100, 300])
@pytest.mark.parametrize("K,F", SHAPES)
def test_products_beyond_fp16(K, F, M, act):
    """dh u act'(g) up to some 1e6, weights small enough for an fp16 dx."""
    lay, wg, wu = _gated(K, F, -6)
    dh, gu = _t(1, M, F, std=100.0), _t(2, M, 2, F)
    gu[:, 1] *= 700
    dh[:, ::3] *= 0.01
    _gated_case(lay, wg, wu, dh, gu, act)
    assert lay.fused_read_error() == 0


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [1, 17, 100, 300])
@pytest.mark.parametrize("K,N", SHAPES)
def test_small_gradients(K, N, M, act):
    """Unscaled gradients near 1e-6, weights of about 1: dz is below fp16's normal range."""
    lay, w = _linear(K, N, 6)
    dy, z = _t(3, M, N, std=2.0 ** -20), _t(4, M, N)
    _linear_case(lay, w, dy, z, act)
    gat, wg, wu = _gated(K, N, 6)
    gu = _t(5, M, 2, N)
    gu[:, 1] *= 2.0 ** -4
    _gated_case(gat, wg, wu, dy, gu, act)
    assert lay.fused_read_error() == 0 and gat.fused_read_error() == 0


@pytest.mark.parametrize("M", [40, 200])
def test_rows_of_different_sizes(M):
    """Every row at its own power of two from 2^-24 to 2^8, a row of zeros among them, and single
    elements of 2^15 in rows of 2^-5."""
    K, N = 256, 1168
    lay, w = _linear(K, N, 0)
    dy, z = _t(6, M, N), _t(7, M, N)
    dy *= (2.0 ** (torch.arange(M, device=DEV) % 33 - 24)).unsqueeze(1).half()
    dy[5] = 0
    dy[7::33] = _t(8, len(dy[7::33]), N, std=2.0 ** -5)
    dy[7::33, 100] = 2.0 ** 15
    z[7::33, 100] = 3.0
    _linear_case(lay, w, dy, z, "gelu")
    assert not lay.linear_backward(dy, z=z, act="gelu")[5].any()


def test_power_of_two_scaling_is_exact():
    """Gradients times 2^k give dx times 2^k bit for bit, as long as dx stays in fp16's normal
    range."""
    K, N, M = 256, 1168, 40
    lay, _ = _linear(K, N, 0)
    dy, z = _t(9, M, N, std=2.0 ** -3), _t(10, M, N)
    dy = (dy.float() * 2 ** 10).round().div(2 ** 10).half()  # exact when made smaller, too
    want = lay.linear_backward(dy, z=z, act="silu").double()
    for k in (-4, -2, 3, 6):
        got = lay.linear_backward((dy.double() * 2.0 ** k).half(), z=z, act="silu").double()
        # (both normal: below 2^-14 fp16 rounds to multiples of 2^-24, which do not scale)
        big = (want.abs() * 2.0 ** k >= 2.0 ** -14) & (want.abs() >= 2.0 ** -14)
        assert torch.equal(got[big], want[big] * 2.0 ** k)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_not_finite_gradients_stay_in_their_row(bad):
    K, N, M = 256, 1168, 40
    lay, _ = _linear(K, N, 0)
    dy, z = _t(11, M, N), _t(12, M, N)
    clean = lay.linear_backward(dy, z=z, act="silu")
    dy[9, 77] = bad
    dx = lay.linear_backward(dy, z=z, act="silu")
    keep = [m for m in range(M) if m != 9]
    assert torch.equal(dx[keep], clean[keep])
    assert not torch.isfinite(dx[9]).all()


@pytest.mark.parametrize("db", [False, True])
def test_infinities_without_a_gradient(db):
    """ReLU at g = -infinity (an overflown gate) passes nothing on; the row's other elements, beyond
    fp16 or far below 1, keep their scaling."""
    K, F, M = 256, 208, 40
    for power, std in ((-6, 100.0), (6, 2.0 ** -20)):
        lay, wg, wu = _gated(K, F, power)
        dh, gu = _t(13, M, F, std=std), _t(14, M, 2, F)
        gu[:, 1] *= 700 if std > 1 else 2.0 ** -4
        clean = gu.clone()
        clean[:, 0, 5::16] = -1.0
        gu[:, 0, 5::16] = float("-inf")
        _gated_case(lay, wg, wu, dh, clean, "relu")
        sums = torch.empty((2, F), dtype=torch.float32, device=DEV) if db else None
        got = lay.backward(dh, gu, act="relu", dbias=sums)
        assert torch.equal(got, lay.backward(dh, clean, act="relu"))
