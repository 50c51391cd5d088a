"""More of the 8-bit floating-point layers without a GPU: refusals of the norm's backward pass where
rows have no expert, of tensors that forward-mode differentiation follows, and of sizes whose products
pass 64 bits."""
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


@pytest.mark.parametrize("E", [0, 1, 1024])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("M,N,K", [(16 * ((1 << 20) - 1), 1 << 30, 1 << 30), (4, 1 << 20, 1 << 20),
                                   (1 << 24, 1 << 30, 1 << 10), (1, 1 << 30, 1 << 30)])
def test_products_of_sizes(M, N, K, backward, E):
    """Blocks of the output, experts, rows and blocks of the sum: 2^66 and 2^76 in the first case."""
    name = ("qlinear_fp8_grouped" if E else "qlinear_fp8_linear") + ("_backward" if backward else "")
    head = (0, P, 2 * P, 7 * P) if E else (0, P, 2 * P)
    rows = (M, E) if E else (M,)
    assert getattr(L, name)(*head, 3 * P, 4 * P, 5 * P, *rows, N, K, 6 * P, 1 << 20, None) == SHAPE


def test_offsets_of_the_norm_are_counted():
    torch = pytest.importorskip("torch")
    from weight_only_quantized_gemv_b200 import layers
    assert layers._MAX_EXPERTS == 1024
    with pytest.raises(ValueError):
        layers.Fp8Experts(torch.zeros(1025, 16, 16, dtype=torch.uint8), torch.ones(1025, 1, 1),
                          device="cpu")


def test_tangents_are_refused():
    torch = pytest.importorskip("torch")
    from torch.autograd import forward_ad
    from weight_only_quantized_gemv_b200 import layers
    plain, seen = torch.randn(4, 32).half(), []

    def checks(t):
        return (lambda: layers._fused_ptr(t, (4, 32), -1, "x", torch.float16),
                lambda: layers._row_ptr(t, -1, "x"))

    class Inside(torch.autograd.Function):
        @staticmethod
        def forward(ctx, a):
            seen.extend(f() for f in checks(a))
            return a.clone()

        @staticmethod
        def jvp(ctx, g):
            return g

    with forward_ad.dual_level():
        dual = forward_ad.make_dual(plain, torch.ones_like(plain))
        for t in (dual, dual.clone(), dual.view(4, 32)):
            for f in checks(t):
                with pytest.raises(ValueError, match="tangent"):
                    f()
        with pytest.raises(ValueError, match="tangent"):
            layers._row_ptr(dual[:, :16], -1, "x")
        for f in checks(plain):
            f()
        Inside.apply(dual)
    assert seen == [plain.data_ptr(), (plain.data_ptr(), 32)]
    for f in checks(plain):
        f()
