"""One workspace for layers of more columns than the fixed part of its counters covers (524288 for
the GEMV, 4194304 for the bias gradient) and for others, on the GPU: the wide layers' further
counters lie where other calls' sums do."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from tests import fp8_ref
    from weight_only_quantized_gemv_b200 import layers

DEV = "cuda:0"


def _w4(K, N, seed):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 2 ** 32, (K // 8, N), dtype=np.uint32)
    scales = (rng.random((K // 128, N)) * 0.01 + 0.01).astype(np.float16)
    zeros = rng.integers(6, 10, (K // 128, N)).astype(np.float16)
    return layers.QuantLinear(ql.QL_FMT_W4, K, N, codes, scales, zeros, device=DEV)


def _fp8(gen):
    """A layer with 4096 rows of weights and the codes of 16 rows: its call leaves parts' sums."""
    lay = layers.Fp8Linear(*fp8_ref.weights(gen, 4096, 4096))
    return lay, *fp8_ref.quantize(torch.randn(16, 4096, generator=gen, device=DEV).double())


def test_gemv_of_a_wide_layer_in_turn_with_others():
    gen = torch.Generator(device=DEV).manual_seed(1)
    K, N = 256, 524288 + 16384
    wide, (f8, q, s) = _w4(K, N, 1), _fp8(gen)
    norm = layers.RMSNorm(torch.ones(2048, dtype=torch.float16, device=DEV))
    t, rstd = torch.randn(200, 2048, device=DEV).half(), torch.rand(200, device=DEV)
    dw = torch.empty(2048, device=DEV)
    ws = max((lay.new_workspace(200, backward=False) for lay in (wide, f8, norm)),
             key=lambda w: w.numel())
    for M in (1, 2, 12, 1):
        x = torch.randn(M, K, generator=gen, device=DEV).half()
        want, want8 = wide.linear(x), f8.forward(q, s)
        for other in ("product", "norm", "product"):
            if other == "product":
                assert torch.equal(f8.forward(q, s, workspace=ws), want8)
            else:
                norm.backward(t, t, rstd, dweight=dw, workspace=ws)
            y = torch.full_like(want, float("nan"))
            assert torch.equal(wide.linear(x, y=y, workspace=ws), want), (M, other)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f8.forward(q, s, workspace=ws)
            wide.linear(x, y=y, workspace=ws)
        for _ in range(2):
            y.fill_(float("nan"))
            graph.replay()
            assert torch.equal(y, want), M
        del graph
    assert ql.qlinear_read_error(ws) == 0


def test_bias_gradient_of_a_wide_layer_in_turn_with_others():
    gen = torch.Generator(device=DEV).manual_seed(2)
    K, N, M = 128, 4194304 + 65536, 70
    wide, (f8, q, s) = _w4(K, N, 2), _fp8(gen)
    dy = (0.01 * torch.randn(M, N, generator=gen, device=DEV)).half()
    ws = max((lay.new_workspace(M) for lay in (wide, f8)), key=lambda w: w.numel())
    dbias, want = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    dx, want8 = wide.linear_backward(dy, dbias=want), f8.forward(q, s)
    for _ in range(2):
        assert torch.equal(f8.forward(q, s, workspace=ws), want8)
        dbias.fill_(float("nan"))
        assert torch.equal(wide.linear_backward(dy, dbias=dbias, workspace=ws), dx)
        assert torch.equal(dbias, want)
    err = dy.abs().sum(0, dtype=torch.double) * (M + 8) * 2.0 ** -24
    assert bool(((want - dy.sum(0, dtype=torch.double)).abs() <= err).all())
    assert ql.qlinear_read_error(ws) == 0
