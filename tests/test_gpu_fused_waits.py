"""Failure detection of the fused layers' bounded waits, on the GPU, without a fault: one wait is
made to run out by a delay that ends by itself, the call returns and the flag is read; after the
workspace has been cleared the next call is bit-identical to one before.

The tensor-core products give up (their outputs are then undefined): both tile forms (one CTA up
to 64 rows, a cluster pair above), whole and split tiles, both directions.  The GEMV with an
epilogue waits on and finishes, as the plain one does.
"""
import pytest

from synth import gen
from tests import fused_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    import weight_only_quantized_gemv_b200 as ql
    yield
    ql.qlinear_debug_wait_test()  # defaults again, whatever the test did


def _layer(seed, K, N):
    from weight_only_quantized_gemv_b200 import layers
    return layers.from_uniform(gen.uniform_layer(seed, K, N, 4), DEV)


def _t(seed, *shape):
    return torch.from_numpy(ref.seeded(seed, *shape)).to(DEV)


# 8 units are split between workers; 9 * 8 row blocks are whole tiles of several workers
@pytest.mark.parametrize("late", ["copy", "mma"])
@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("K,N", [(1024, 1168), (1152, 18944)])
@pytest.mark.parametrize("M", [20, 60, 100, 300])
def test_product_gives_up(M, K, N, backward, late):
    import weight_only_quantized_gemv_b200 as ql
    lay = _layer(70, K, N)
    x = _t(1, M, N if backward else K)
    call = lay.linear_backward if backward else lay.linear
    want = call(x)
    assert lay.fused_read_error() == 0
    ql.qlinear_debug_wait_test(2000, 10000 if late == "copy" else 0,
                               10000 if late == "mma" else 0)
    call(x)
    torch.cuda.synchronize()
    flags = lay.fused_read_error()
    assert flags, "the late step was not reported"
    ql.qlinear_debug_wait_test()
    for _ in range(3):
        assert torch.equal(call(x), want)
    assert lay.fused_read_error() == 0


@pytest.mark.parametrize("M", [1, 12])
def test_gemv_with_epilogue_reports_a_late_copy(M):
    import weight_only_quantized_gemv_b200 as ql
    lay = _layer(71, 1024, 256)
    x, res = _t(2, M, 1024), _t(3, M, 256)
    want = lay.linear(x, residual=res, act="silu")
    assert lay.fused_read_error() == 0
    ql.qlinear_debug_wait_test(1, 5000, 0)
    got = lay.linear(x, residual=res, act="silu")
    torch.cuda.synchronize()
    assert lay.fused_read_error() & 1
    assert torch.equal(got, want)  # the second wait let the copy land
    ql.qlinear_debug_wait_test()
    assert torch.equal(lay.linear(x, residual=res, act="silu"), want)
    assert lay.fused_read_error() == 0


@pytest.mark.parametrize("fmt,M", [("w4", 200), ("w8", 200), ("w8", 60), ("w8", 100),
                                   ("lut4", 300)])
@pytest.mark.parametrize("backward", [False, True])
def test_no_flag_behind_a_long_kernel(fmt, M, backward):
    """A call that starts early, on SMs that the kernel before it leaves idle, waits for that
    kernel as long as it takes: the limit of its own waits begins after it."""
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers
    K, N = 2048, 2320
    if fmt == "lut4":
        lay = layers.from_lut4(gen.lut4_layer(72, K, N), DEV)
    else:
        lay = layers.from_uniform(gen.uniform_layer(72, K, N, int(fmt[1:])), DEV)
    small = _layer(73, 128, 16)
    x, xs = _t(4, M, N if backward else K), _t(5, 20, 128)
    call = lay.linear_backward if backward else lay.linear
    want, first = call(x), small.linear(xs)
    for one in (lay, small):
        assert one.fused_read_error() == 0
    ql.qlinear_debug_wait_test(1000000, 60000, 0)  # one CTA, for 60 ms
    out = small.linear(xs)
    ql.qlinear_debug_wait_test(5000, 0, 0)
    got = call(x)
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(got, want)
    for one in (lay, small):
        assert one.fused_read_error() == 0


def test_limit_grows_with_the_tile():
    """The epilogue waits for a whole tile: 1024 units of about 0.45 us against a limit of 1 us
    and 4 us a unit.  (148 tiles of 128 columns: every worker has one, and none is shared.)"""
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers
    K, N, M = 131072, 18944, 20
    q = torch.randint(0, 256, (K * N // 4,), dtype=torch.uint8, device=DEV)
    p0 = torch.full((K // 128 * N,), 2.0 ** -10, dtype=torch.float16, device=DEV)
    p1 = torch.ones(K // 128 * N, dtype=torch.float16, device=DEV)
    x, y = _t(6, M, K), torch.empty((M, N), dtype=torch.float16, device=DEV)
    ws = torch.zeros(ql.qlinear_fused_workspace_bytes(2, M, N, K, False), dtype=torch.uint8,
                     device=DEV)
    ql.qlinear_linear(2, x, q, p0, p1, y, M, N, K, ws)
    want = y.clone()
    ql.qlinear_debug_wait_test(1, 0, 0)
    ql.qlinear_linear(2, x, q, p0, p1, y, M, N, K, ws)
    torch.cuda.synchronize()
    assert ql.qlinear_read_error(ws) == 0
    assert torch.equal(y, want) and bool(torch.isfinite(y).all())
