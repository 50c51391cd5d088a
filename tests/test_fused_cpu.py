"""The fused linear layers without a GPU: packers, and refusals before the device is touched."""
import numpy as np
import pytest

import weight_only_quantized_gemv_b200 as ql

FMTS = [2, 4, 8, 16]
P = 4096  # stands for an aligned device pointer; never followed


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K,F", [(128, 16), (384, 208), (256, 144)])
def test_gated_packing_is_packing_of_alternating_tiles(fmt, K, F):
    rs = np.random.default_rng(fmt + F)
    bits = 4 if fmt == 16 else fmt
    if fmt == 16:
        mats = [rs.integers(0, 256, (K // 2, F), dtype=np.uint8) for _ in range(2)]
        pars = [rs.standard_normal((K // 64, F)).astype(np.float32) for _ in range(2)]
    else:
        mats = [rs.integers(0, 2 ** 32, (K * bits // 32, F), dtype=np.uint32) for _ in range(2)]
        pars = [rs.standard_normal((K // 128, F)).astype(np.float16) for _ in range(2)]

    def interleave(a, b):
        r = a.shape[0]
        return np.stack([a.reshape(r, F // 16, 16), b.reshape(r, F // 16, 16)], 2).reshape(r, 2 * F)

    assert np.array_equal(ql.qlinear_pack_gated(fmt, *mats, F, K),
                          ql.qlinear_pack(fmt, interleave(*mats), 2 * F, K))
    assert np.array_equal(ql.qlinear_pack_params_gated(fmt, *pars, F, K),
                          ql.qlinear_pack_params(fmt, interleave(*pars), 2 * F, K).reshape(-1))


def test_gated_packing_refusals():
    a = np.zeros((16, 32), dtype=np.uint32)
    with pytest.raises(ql.QLinearError):
        ql.qlinear_pack_gated(4, a, a[:8], 32, 128)
    with pytest.raises(ql.QLinearError):
        ql.qlinear_pack_gated(4, a, a, 40, 128)
    with pytest.raises(ql.QLinearError):
        ql.qlinear_pack_gated(3, a, a, 32, 128)
    assert ql._lib.qlinear_pack_gated(4, None, P, P, 32, 128) == 1
    assert ql._lib.qlinear_pack_params_gated(4, P, None, P, 32, 128) == 1
    assert ql._lib.qlinear_pack_gated(4, P, P, P, (1 << 29) + 16, 128) == 2


def _linear(fmt=4, x=P, w=P * 1000, p0=P * 2000, p1=P * 3000, bias=None, res=None, act=0,
            y=P * 4000, z=None, M=4, N=64, K=128, ws=P * 5000, nbytes=1 << 20):
    return ql._lib.qlinear_linear(fmt, x, w, p0, p1, bias, res, act, y, z, M, N, K, ws, nbytes,
                                  None)


def _gated(fmt=4, x=P, w=P * 1000, p0=P * 2000, p1=P * 3000, bias=None, act=4, h=P * 4000,
           gu=None, M=4, F=64, K=128, ws=P * 5000, nbytes=1 << 20):
    return ql._lib.qlinear_gated(fmt, x, w, p0, p1, bias, act, h, gu, M, F, K, ws, nbytes, None)


def _linear_bwd(fmt=4, dy=P, z=P * 500, w=P * 1000, p0=P * 2000, p1=P * 3000, act=4,
                dx=P * 4000, db=None, M=4, N=64, K=128, ws=P * 5000, nbytes=1 << 20):
    return ql._lib.qlinear_linear_backward(fmt, dy, z, w, p0, p1, act, dx, db, M, N, K, ws,
                                           nbytes, None)


def _gated_bwd(fmt=4, dh=P, gu=P * 500, w=P * 1000, p0=P * 2000, p1=P * 3000, act=4,
               dx=P * 4000, db=None, M=4, F=64, K=128, ws=P * 5000, nbytes=1 << 20):
    return ql._lib.qlinear_gated_backward(fmt, dh, gu, w, p0, p1, act, dx, db, M, F, K, ws,
                                          nbytes, None)


NULL, SHAPE, ALIGN, UNSUPPORTED, ALIAS = 1, 2, 3, 4, 8
ENTRIES = [_linear, _gated, _linear_bwd, _gated_bwd]


@pytest.mark.parametrize("call", ENTRIES)
def test_common_refusals(call):
    assert call(fmt=3) == UNSUPPORTED and call(fmt=32) == UNSUPPORTED
    assert call(act=5) == UNSUPPORTED and call(act=-1) == UNSUPPORTED
    for arg in ("w", "p0", "p1"):
        assert call(**{arg: None}) == NULL
    for M in (0, -1, (1 << 24) + 1):
        assert call(M=M) == SHAPE
    for K in (0, 64, 130, -128):
        assert call(K=K) == SHAPE
    width = "N" if call in (_linear, _linear_bwd) else "F"
    for n in (0, 8, 24, -16, (1 << 30) + 16, 2 ** 31 - 16):
        assert call(**{width: n}) == SHAPE
    assert call(K=(1 << 30) + 128) == SHAPE
    assert call(w=P * 1000 + 16) == ALIGN
    assert call(p0=P * 2000 + 2) == ALIGN and call(p1=P * 3000 + 8) == ALIGN
    assert call(fmt=16, p0=P * 2000 + 1) == ALIGN


def test_pointer_refusals():
    assert _linear(x=None) == NULL and _linear(y=None) == NULL
    assert _gated(x=None) == NULL and _gated(h=None) == NULL
    assert _linear_bwd(dy=None) == NULL and _linear_bwd(dx=None) == NULL
    assert _linear_bwd(z=None) == NULL
    assert _gated_bwd(gu=None, act=0) == NULL
    for arg in ("x", "y", "z", "bias", "res"):
        assert _linear(**{arg: P * 4500 + 8}) == ALIGN
    for arg in ("x", "h", "gu", "bias"):
        assert _gated(**{arg: P * 4500 + 8}) == ALIGN
    for arg in ("dy", "z", "dx", "db"):
        assert _linear_bwd(**{arg: P * 4500 + 8}) == ALIGN


def test_overlaps_are_refused():
    y = P * 4000
    # one byte range inside another counts, neighbours do not
    assert _linear(x=y) == ALIAS
    assert _linear(x=y - 4 * 128 * 2 + 16) == ALIAS
    assert _linear(z=y + 16) == ALIAS
    assert _linear(bias=y) == ALIAS
    assert _linear(res=y + 16) == ALIAS
    assert _linear(w=y) == ALIAS and _linear(ws=y) == ALIAS and _linear(x=P * 5000) == ALIAS
    assert _gated(x=y) == ALIAS and _gated(gu=y) == ALIAS
    assert _linear_bwd(dy=y) == ALIAS and _linear_bwd(z=y) == ALIAS and _linear_bwd(db=y) == ALIAS
    assert _gated_bwd(dh=y) == ALIAS and _gated_bwd(gu=y) == ALIAS and _gated_bwd(ws=y) == ALIAS
    # (an exact residual alias and a neighbour get as far as the device or the workspace)
    assert _linear(res=y, nbytes=0, ws=None) not in (ALIAS, 0)
    assert _linear(z=y + 4 * 64 * 2, nbytes=0, ws=None) not in (ALIAS, 0)


def test_workspace_query_refuses_bad_arguments():
    for args in ((3, 1, 64, 128), (4, 0, 64, 128), (4, 1, 60, 128), (4, 1, 64, 100)):
        assert ql.qlinear_fused_workspace_bytes(*args) == 0


def test_unknown_activation_name():
    with pytest.raises(ql.QLinearError):
        ql._act("swish")


def test_short_tables_are_refused():
    """The kernels read 16 entries of a LUT4 table, whatever it holds."""
    pytest.importorskip("torch")
    from synth import gen
    from weight_only_quantized_gemv_b200 import layers
    lt = gen.lut4_layer(1, 128, 16)
    good, bad = (lt.qbytes, lt.lut, lt.absmax), (lt.qbytes, lt.lut[:8], lt.absmax)
    for args in ((bad, bad), (good, bad), (bad, good)):
        with pytest.raises(ValueError, match="16 entries"):
            layers.GatedLinear(ql.QL_FMT_LUT4, 128, 16, *args, device="cpu")
    assert layers.GatedLinear(ql.QL_FMT_LUT4, 128, 16, good, good, device="cpu").p0.numel() == 16
    with pytest.raises(ValueError, match="16 entries"):
        layers.QuantLinear(ql.QL_FMT_LUT4, 128, 16, *bad, device="cpu")
