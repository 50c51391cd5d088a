"""Bounded waits of the e4m3 products that run out, on the GPU: single CTAs with rows as the A operand,
and every kernel with the experts' offsets."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from tests import fp8_ref as ref
    from weight_only_quantized_gemv_b200 import layers

SHAPES = [(1024, 1168), (1152, 18944)]


@pytest.fixture(autouse=True)
def _defaults():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    yield
    ql.qlinear_debug_wait_test()  # whatever the test did


def _gives_up(lay, call, late):
    """A late step of the first worker is reported; afterwards calls are right again."""
    want = call()
    assert lay.fused_read_error() == 0
    ql.qlinear_debug_wait_test(2000, 10000 if late == "copy" else 0, 10000 if late == "mma" else 0)
    call()
    torch.cuda.synchronize()
    assert lay.fused_read_error(), "the late step was not reported"
    ql.qlinear_debug_wait_test()
    for _ in range(3):
        assert torch.equal(call(), want)
    assert lay.fused_read_error() == 0


def _codes(gen, M, C):
    return ref.quantize(torch.randn(M, C, generator=gen, device="cuda").double())


@pytest.mark.parametrize("late", ["copy", "mma"])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("N,K", SHAPES)
def test_single_ctas(N, K, backward, late):
    gen = torch.Generator(device="cuda").manual_seed(N)
    lay = layers.Fp8Linear(*ref.weights(gen, N, K))
    q, s = _codes(gen, 100, N if backward else K)
    _gives_up(lay, lambda: (lay.backward if backward else lay.forward)(q, s), late)


@pytest.mark.parametrize("late", ["copy", "mma"])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("M", [30, 80, 150, 500, 1200])
def test_by_expert(M, N, K, backward, late):
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    lay = layers.Fp8Experts(*ref.weights(gen, 3, N, K))
    q, s = _codes(gen, M, N if backward else K)
    at = torch.tensor([3, M // 2, M // 2, M - 5], dtype=torch.int32, device="cuda")

    def call():
        out = torch.zeros(M, K if backward else N, dtype=torch.bfloat16, device="cuda")
        return (lay.backward if backward else lay.forward)(q, s, at, out)

    _gives_up(lay, call, late)
