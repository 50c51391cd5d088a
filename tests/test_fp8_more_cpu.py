"""More of the 8-bit floating-point layers without a GPU: refusals of the norm's backward pass where
rows have no expert."""
import pytest

import weight_only_quantized_gemv_b200 as ql

P = 1 << 24  # stands for an aligned device pointer; never followed
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8
L = ql._lib


def _norm_bwd(t=0, dy=P, x=2 * P, rstd=3 * P, w=5 * P, dt=6 * P, off=10 * P, dx=7 * P, dw=8 * P, M=4,
              E=3, K=256, ws=9 * P, nbytes=1 << 20):
    return L.qlinear_rmsnorm_backward_grouped(t, dy, x, rstd, w, dt, off, dx, dw, M, E, K, ws,
                                              nbytes, None)


def test_norm_backward_by_expert_refusals():
    for t in (-1, 2):
        assert _norm_bwd(t=t) == UNSUPPORTED
    for M in (0, -1, (1 << 24) + 1):
        assert _norm_bwd(M=M) == SHAPE
    for E in (0, -1, 1025):
        assert _norm_bwd(E=E) == SHAPE
    for K in (0, 8, 24, 250, -16, 32784):
        assert _norm_bwd(K=K) == SHAPE
    for a in ("dy", "x", "rstd", "w", "off", "dx"):
        assert _norm_bwd(**{a: None}) == NULL
    for a in ("dy", "x", "w", "dt", "dx"):
        assert _norm_bwd(**{a: 20 * P + 8}) == ALIGN
    for a in ("rstd", "off", "dw"):
        assert _norm_bwd(**{a: 20 * P + 2}) == ALIGN


def test_offsets_of_the_norm_are_counted():
    torch = pytest.importorskip("torch")
    from weight_only_quantized_gemv_b200 import layers
    assert layers._MAX_EXPERTS == 1024
    with pytest.raises(ValueError):
        layers.Fp8Experts(torch.zeros(1025, 16, 16, dtype=torch.uint8), torch.ones(1025, 1, 1),
                          device="cpu")
