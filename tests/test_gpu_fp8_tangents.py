"""Tensors that forward-mode differentiation follows are refused by the layers, on the GPU."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from tests import fp8_ref as ref
    from torch.autograd import forward_ad
    from weight_only_quantized_gemv_b200 import layers


def test_tangents_are_refused():
    M, K = 3, 256
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, r = (ref.activations(gen, M, K, torch.float16) for _ in range(2))
    rstd = torch.ones(M, device="cuda")
    norm = layers.RMSNorm(torch.ones(K, dtype=torch.float16, device="cuda"))
    f8 = layers.Fp8Linear(*ref.weights(gen, 64, K))
    w4 = layers.QuantLinear(ql.QL_FMT_W4, K, 64, np.zeros((K // 8, 64), np.uint32),
                            np.ones((2, 64), np.float16), np.zeros((2, 64), np.float16))
    q, s = layers.fp8_quantize(x)
    with forward_ad.dual_level():
        d = forward_ad.make_dual(x, torch.ones_like(x))
        ds = forward_ad.make_dual(s, torch.ones_like(s))
        for call in (lambda: layers.fp8_quantize(d), lambda: layers.fp8_quantize(d[:, :128]),
                     lambda: layers.fp8_gated(d), lambda: layers.fp8_gated_backward(d[:, :128], r),
                     lambda: layers.fp8_quantize_weights(torch.cat([d] * 16)),
                     lambda: norm.forward(d), lambda: norm.forward(x, d),
                     lambda: norm.backward(d, x, rstd), lambda: norm.backward(x, d, rstd),
                     lambda: f8.forward(q, ds), lambda: w4.linear(d),
                     lambda: w4.linear(x, residual=d[:, :64].contiguous())):
            with pytest.raises(ValueError, match="tangent"):
                call()
        again = layers.fp8_quantize(x)
    assert torch.equal(again[0].view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(again[1], s)
