"""The 8-bit floating-point layers without a GPU: refusals before the device is touched, and the
checks of the layers' arguments."""
import pytest

import weight_only_quantized_gemv_b200 as ql

P = 1 << 24  # stands for an aligned device pointer; never followed
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 8
L = ql._lib


def _quantize(t=0, x=P, ldx=256, q=2 * P, s=3 * P, M=4, K=256):
    return L.qlinear_fp8_quantize(t, x, ldx, q, s, M, K, None)


def _weights(t=0, x=P, q=2 * P, s=3 * P, E=2, M=64, K=256):
    return L.qlinear_fp8_quantize_weights(t, x, q, s, E, M, K, None)


def _gated(t=0, act=4, x=P, q=2 * P, s=3 * P, M=4, K=256):
    return L.qlinear_fp8_gated(t, act, x, q, s, M, K, None)


def _gated_bwd(t=0, act=4, dh=4 * P, x=P, q=2 * P, s=3 * P, M=4, K=256):
    return L.qlinear_fp8_gated_backward(t, act, dh, x, q, s, M, K, None)


def _norm(t=0, x=P, ldx=256, r=4 * P, w=5 * P, eps=1e-6, total=6 * P, y=7 * P, q=2 * P, s=3 * P,
          rstd=8 * P, M=4, K=256):
    return L.qlinear_rmsnorm(t, x, ldx, r, w, eps, total, y, q, s, rstd, M, K, None)


def _norm_bwd(t=0, dy=P, x=2 * P, rstd=3 * P, w=5 * P, dt=6 * P, dx=7 * P, dw=8 * P, M=4, K=256,
              ws=9 * P, nbytes=1 << 20):
    return L.qlinear_rmsnorm_backward(t, dy, x, rstd, w, dt, dx, dw, M, K, ws, nbytes, None)


def _linear(t=0, q=P, s=2 * P, w=3 * P, sw=4 * P, y=5 * P, M=4, N=64, K=256, ws=6 * P,
            nbytes=1 << 20, entry=L.qlinear_fp8_linear):
    return entry(t, q, s, w, sw, y, M, N, K, ws, nbytes, None)


def _linear_bwd(**kw):
    return _linear(entry=L.qlinear_fp8_linear_backward, **kw)


def _grouped(t=0, q=P, s=2 * P, off=7 * P, w=3 * P, sw=4 * P, y=5 * P, M=4, E=3, N=64, K=256,
             ws=6 * P, nbytes=1 << 20, entry=L.qlinear_fp8_grouped):
    return entry(t, q, s, off, w, sw, y, M, E, N, K, ws, nbytes, None)


def _grouped_bwd(**kw):
    return _grouped(entry=L.qlinear_fp8_grouped_backward, **kw)


PRODUCTS = [_linear, _linear_bwd, _grouped, _grouped_bwd]
ROWS = [_quantize, _gated, _gated_bwd, _norm, _norm_bwd] + PRODUCTS


@pytest.mark.parametrize("call", ROWS + [_weights])
def test_common_refusals(call):
    for t in (-1, 2):
        assert call(t=t) == UNSUPPORTED
    if call is not _weights:
        for M in (0, -1, (1 << 24) + 1):
            assert call(M=M) == SHAPE
    for K in (0, 8, 24, 250, -16, (1 << 30) + 16):
        assert call(K=K) == SHAPE


@pytest.mark.parametrize("call", [_gated, _gated_bwd])
def test_unknown_activations(call):
    assert call(act=5) == UNSUPPORTED and call(act=-1) == UNSUPPORTED
    assert call(K=(1 << 29) + 16) == SHAPE


@pytest.mark.parametrize("call,args,align", [
    (_quantize, "xqs", 16), (_weights, "xqs", 16), (_gated, "xqs", 16),
    (_gated_bwd, ("dh", "x", "q", "s"), 16)])
def test_pointers_of_codes(call, args, align):
    for a in args:
        assert call(**{a: None}) == NULL
        assert call(**{a: 10 * P + 2}) == ALIGN
    assert call(q=10 * P + 8) == ALIGN and call(x=10 * P + 8) == ALIGN
    assert call(s=10 * P + 4, x=10 * P) == ALIAS   # scales inside x


def test_strided_rows():
    assert _quantize(ldx=255) == SHAPE and _quantize(ldx=260) == ALIGN
    assert _norm(ldx=128) == SHAPE and _norm(ldx=257) == ALIGN
    # the rows in between count as x's: an output there is refused
    assert _quantize(ldx=1 << 20, q=P + (1 << 20)) == ALIAS


def test_norm_refusals():
    assert _norm(x=None) == NULL and _norm(w=None) == NULL
    assert _norm(q=None, s=None, y=None) == NULL     # no output
    assert _norm(q=None) == NULL and _norm(s=None) == NULL
    assert _norm(K=32784, ldx=32784) == SHAPE
    for eps in (-1.0, float("nan")):
        assert _norm(eps=eps) == SHAPE
    for a in ("x", "r", "w", "total", "y", "q"):
        assert _norm(**{a: 20 * P + 8}) == ALIGN
    assert _norm(rstd=20 * P + 2) == ALIGN and _norm(s=20 * P + 2) == ALIGN
    for out in ("y", "q", "s", "rstd"):
        for other in (P, 4 * P, 5 * P, 6 * P):
            assert _norm(**{out: other}) == ALIAS
    # the stream is updated in place or not at all
    assert _norm(total=P + 16) == ALIAS and _norm(total=4 * P + 16) == ALIAS
    assert _norm(total=P, ldx=512) == ALIAS
    assert _norm(total=5 * P) == ALIAS


def test_norm_backward_refusals():
    for a in ("dy", "x", "rstd", "w", "dx"):
        assert _norm_bwd(**{a: None}) == NULL
    for a in ("dy", "x", "w", "dt", "dx"):
        assert _norm_bwd(**{a: 20 * P + 8}) == ALIGN
    assert _norm_bwd(K=32784) == SHAPE


@pytest.mark.parametrize("call", PRODUCTS)
def test_product_refusals(call):
    for a in ("q", "s", "w", "sw", "y"):
        assert call(**{a: None}) == NULL
        assert call(**{a: 20 * P + 2}) == ALIGN
    for a in ("q", "w", "y"):
        assert call(**{a: 20 * P + 8}) == ALIGN
    for N in (0, 8, 30, -16, (1 << 30) + 16):
        assert call(N=N) == SHAPE
    assert call(ws=None) == WORKSPACE and call(nbytes=1024) == WORKSPACE
    assert call(ws=6 * P + 16) == ALIGN
    for a in ("q", "s", "w", "sw", "ws"):
        assert call(**{a: 5 * P}) == ALIAS
    assert call(q=6 * P) == ALIAS


@pytest.mark.parametrize("call", [_grouped, _grouped_bwd])
def test_grouped_refusals(call):
    assert call(off=None) == NULL and call(off=20 * P + 2) == ALIGN
    for E in (0, -1, 1025):
        assert call(E=E) == SHAPE
    assert call(off=5 * P) == ALIAS


def test_workspace_queries_refuse_bad_arguments():
    for args in ((0, 1, 64, 128), (1, 0, 64, 128), (1, 1025, 64, 128), (1, 1, 60, 128),
                 (1, 1, 64, 100)):
        assert ql.qlinear_fp8_workspace_bytes(*args) == 0
    for args in ((0, 128), (1, 24), (1, 32784)):
        assert ql.qlinear_rmsnorm_workspace_bytes(*args) == 0


def test_unknown_type_name():
    with pytest.raises(ql.QLinearError):
        ql._type("float32")
    assert ql._type("bfloat16") == 1 and ql._type(0) == 0


def test_weights_are_checked():
    torch = pytest.importorskip("torch")
    from weight_only_quantized_gemv_b200 import layers
    codes, scales = torch.zeros(48, 144, dtype=torch.uint8), torch.ones(1, 2)
    lay = layers.Fp8Linear(codes, scales, device="cpu")
    assert (lay.N, lay.K, lay.codes.dtype) == (48, 144, torch.float8_e4m3fn)
    assert lay.weight_bytes == 48 * 144 + 8
    assert layers.Fp8Linear(codes.numpy(), scales.numpy(), device="cpu").K == 144
    for c, s in ((codes, torch.ones(2, 2)), (codes.float(), scales), (codes, scales.double()),
                 (codes[None], scales[None])):
        with pytest.raises(ValueError):
            layers.Fp8Linear(c, s, device="cpu")
    for shape in ((40, 128), (48, 120), (0, 128), (1025, 16, 16)):  # not multiples of 16, too many
        with pytest.raises(ValueError):
            (layers.Fp8Linear if len(shape) == 2 else layers.Fp8Experts)(
                torch.zeros(shape, dtype=torch.uint8),
                torch.ones(*shape[:-2], -(-shape[-2] // 128), 1), device="cpu")
    for rows, columns in ((2 ** 24 + 1, 16), (1, 2 ** 30 + 16), (2 ** 32 + 1, 16)):
        with pytest.raises(ValueError):
            layers._check_size(rows, columns)
    with pytest.raises(ValueError):
        layers.Fp8Experts(codes, scales, device="cpu")
    experts = layers.Fp8Experts(codes[None], scales[None], device="cpu")
    assert experts.E == 1
    with pytest.raises(ValueError):
        layers.Fp8GatedMLP(lay, experts)
    with pytest.raises(ValueError):
        layers.RMSNorm(torch.ones(16))
    for f in (layers.fp8_quantize, layers.fp8_gated):
        with pytest.raises(ValueError):
            f(torch.ones(2, 32))
    with pytest.raises(ValueError):
        layers.fp8_quantize_weights(torch.ones(16, 16))


def test_run_fp8_helpers():
    pytest.importorskip("torch")
    from weight_only_quantized_gemv_b200 import run_fp8
    at = run_fp8.ragged_offsets(100, 8)
    assert at[0] == 0 and at[-1] == 100 and sorted(at) == at and at[3] == at[4]
    assert run_fp8.ragged_offsets(7, 1) == [0, 7]
    assert run_fp8.moved_bytes("quantize", 2, 0, 256) == 2 * 2 * 256 + 2 * 256 + 4 * 2 * 2
    assert run_fp8.moved_bytes("linear", 3, 144, 256) == 144 * 256 + 16 + 3 * 256 + 24 + 2 * 3 * 144
