"""The fused linear layers on the GPU: bias / activation / residual epilogue, the gated
projection, and the backward passes, against the fp64 definition with elementwise bounds
(tests/fused_ref.py)."""
import functools

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
FMTS = ["w2", "w4", "w8", "lut4"]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# rows on both sides of every switch: the GEMV's buckets (1, 8, 16), the token tiles
ROWS = [1, 2, 8, 9, 16, 17, 33, 64, 65, 100, 128, 129, 256, 257, 300]
SHAPES = [(128, 16), (384, 208), (1024, 512), (2048, 1168)]


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


@functools.lru_cache(maxsize=32)
def _raw(fmt, K, N, seed):
    lay = gen.lut4_layer(seed, K, N) if fmt == "lut4" else gen.uniform_layer(seed, K, N,
                                                                          int(fmt[1:]))
    return lay, torch.from_numpy(ref.weight(lay, fmt)).to(DEV)


@functools.lru_cache(maxsize=32)
def _linear(fmt, K, N, seed=1):
    lay, w = _raw(fmt, K, N, seed)
    return layers.QuantLinear(ql.FORMATS[fmt], K, N, *ref.canonical(lay, fmt), device=DEV), w


@functools.lru_cache(maxsize=32)
def _gated(fmt, K, F, seed=2):
    (a, wa), (b, wb) = _raw(fmt, K, F, seed), _raw(fmt, K, F, seed + 1)
    ga, up = ref.canonical(a, fmt), ref.canonical(b, fmt)
    if fmt == "lut4":  # one table: the up projection's codes read through the gate's
        b.lut = a.lut
        up = ref.canonical(b, fmt)
        wb = torch.from_numpy(ref.weight(b, fmt)).to(DEV)
    return layers.GatedLinear(ql.FORMATS[fmt], K, F, ga, up, device=DEV), wa, wb


def _t(seed, *shape, std=1.0):
    return torch.from_numpy(ref.seeded(seed, *shape, std=std)).to(DEV)


def _clean(*lays):
    for lay in lays:
        assert lay.fused_read_error() == 0, "a device wait ran out"


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_linear(fmt, K, N, M):
    lay, w = _linear(fmt, K, N)
    i = M + K + N
    act = ACTS[i % 5]
    x, bias, res = _t(i, M, K), _t(i + 1, N, std=0.3), _t(i + 2, M, N)
    bias, res = (bias if i % 2 else None), (res if (i // 2) % 2 else None)
    z = torch.empty((M, N), dtype=torch.float16, device=DEV) if i % 3 else None
    y = lay.linear(x, bias=bias, residual=res, act=act, z=z)
    wy, wz = ref.linear(x.double(), w, None if bias is None else bias.double(),
                        None if res is None else res.double(), act)
    ref.check(y, wy, "y")
    if z is not None:
        ref.check(z, wz, "z")
    _clean(lay)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [3, 40])
def test_linear_every_option(act, M):
    lay, w = _linear("w4", 384, 208)
    x, bias, res = _t(5, M, 384), _t(6, 208, std=0.3), _t(7, M, 208)
    for b in (None, bias):
        for r in (None, res):
            z = torch.empty((M, 208), dtype=torch.float16, device=DEV)
            y = lay.linear(x, bias=b, residual=r, act=act, z=z)
            wy, wz = ref.linear(x.double(), w, None if b is None else b.double(),
                                None if r is None else r.double(), act)
            ref.check(y, wy, f"y {b is None} {r is None}")
            ref.check(z, wz, "z")
    _clean(lay)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K,F", [(128, 16), (384, 208), (1024, 256), (2048, 592)])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated(fmt, K, F, M):
    lay, wg, wu = _gated(fmt, K, F)
    i = M + K + F
    act = ACTS[1 + i % 4]
    x, bias = _t(i, M, K), (_t(i + 1, 2, F, std=0.3) if i % 2 else None)
    gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV) if i % 3 else None
    h = lay.forward(x, bias=bias, act=act, gu=gu)
    wh, wgu = ref.gated(x.double(), wg, wu, None if bias is None else bias.double(), act)
    ref.check(h, wh, "h")
    if gu is not None:
        ref.check(gu, wgu, "gu")
    _clean(lay)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("fmt", FMTS)
def test_linear_backward(fmt, K, N, M):
    lay, w = _linear(fmt, K, N)
    i = M + K + N
    act = ACTS[i % 5]
    dy, z = _t(i, M, N, std=0.25), _t(i + 1, M, N)
    db = torch.empty(N, dtype=torch.float32, device=DEV) if i % 2 else None
    dx = lay.linear_backward(dy, z=None if act == "none" else z, act=act, dbias=db)
    wdx, wdb = ref.linear_backward(dy.double(), z.double(), w, act)
    ref.check(dx, wdx, "dx")
    if db is not None:
        ref.check(db, wdb, "dbias")
    _clean(lay)


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("K,F", [(128, 16), (384, 208), (1024, 256), (2048, 592)])
@pytest.mark.parametrize("fmt", FMTS)
def test_gated_backward(fmt, K, F, M):
    lay, wg, wu = _gated(fmt, K, F)
    i = M + K + F
    act = ACTS[i % 5]
    dh, gu = _t(i, M, F, std=0.25), _t(i + 1, M, 2, F)
    db = torch.empty((2, F), dtype=torch.float32, device=DEV) if i % 2 else None
    dx = lay.backward(dh, gu, act=act, dbias=db)
    wdx, wdb = ref.gated_backward(dh.double(), gu.double(), wg, wu, act)
    ref.check(dx, wdx, "dx")
    if db is not None:
        ref.check(db, wdb, "dbias")
    _clean(lay)


@pytest.mark.parametrize("M", [700, 1500])
@pytest.mark.parametrize("fmt", ["w4", "lut4"])
def test_many_rows(fmt, M):
    """Several waves of tiles per worker, then tiles shared between workers."""
    K, F = 1024, 2064
    lay, wg, wu = _gated(fmt, K, F)
    x = _t(M, M, K)
    gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV)
    ref.check(lay.forward(x, gu=gu), ref.gated(x.double(), wg, wu)[0], "h")
    dh = _t(M + 1, M, F, std=0.25)
    db = torch.empty((2, F), dtype=torch.float32, device=DEV)
    wdx, wdb = ref.gated_backward(dh.double(), gu.double(), wg, wu, "silu")
    ref.check(lay.backward(dh, gu, dbias=db), wdx, "dx")
    ref.check(db, wdb, "dbias")
    _clean(lay)


@pytest.mark.parametrize("M", [1, 5, 12, 64, 200])
def test_one_hot(M):
    """x one-hot: the pre-activation is one weight, exact before its rounding to fp16."""
    K, N = 384, 208
    for fmt in FMTS:
        lay, w = _linear(fmt, K, N)
        ks = [(37 * m + 5) % K for m in range(M)]
        x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
        x[torch.arange(M), ks] = 1
        y = lay.linear(x)
        if M > 16 and fmt == "lut4":  # fp16 weights: rounded to fp32 first
            want = w[ks].float().half()
        else:
            want = w[ks].half() if fmt != "lut4" else None
        if want is not None:
            assert torch.equal(y, want), fmt


@pytest.mark.parametrize("M", [1, 16, 48, 300])
def test_gradient_against_differences(M):
    """<dx, v> against central differences of the fp64 forward along v."""
    K, F = 384, 208
    lay, wg, wu = _gated("w4", K, F)
    lin, w = _linear("w8", K, F)
    x, v, dy = _t(1, M, K).double(), _t(2, M, K).double(), _t(3, M, F, std=0.25)
    eps = 1e-4
    for act in ("gelu", "gelu_tanh", "silu"):
        def fwd_gated(xx):
            return (ref.act(act, xx @ wg) * (xx @ wu) * dy.double()).sum()

        def fwd_linear(xx):
            return (ref.act(act, xx @ w) * dy.double()).sum()

        gu = torch.stack([x @ wg, x @ wu], 1).half()
        for dx, fwd in ((lay.backward(dy, gu, act=act), fwd_gated),
                        (lin.linear_backward(dy, (x @ w).half(), act=act), fwd_linear)):
            want = float(fwd(x + eps * v) - fwd(x - eps * v)) / (2 * eps)
            got = float((dx.double() * v).sum())
            # |<dx - dx_ref, v>|: REL of |dx| in each direction, independent of v, plus the
            # kept values' rounding
            scale = float(dx.double().norm() * v.norm())
            assert abs(got - want) <= 2 * ref.REL * scale, (act, got, want)


@pytest.mark.parametrize("M", [1, 7, 33, 260])
def test_feed_forward_block(M):
    """Forward and backward of the whole block, as a training step and a decoder run it."""
    K, F = 512, 1152
    gate_up, wg, wu = _gated("w4", K, F)
    down, wd = _linear("w8", F, K, seed=9)
    mlp = layers.GatedMLP(gate_up, down)
    x, dy = _t(1, M, K), _t(2, M, K, std=0.25)
    gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV)
    y = mlp.forward(x, residual=x, gu=gu)
    xd = x.double().requires_grad_(True)
    want = (ref.act("silu", xd @ wg) * (xd @ wu)) @ wd + xd.detach()
    assert float((y.double() - want.detach()).norm()) <= 3 * ref.REL * float(want.detach().norm())
    grad = torch.autograd.grad(want, xd, dy.double())[0]
    dx = mlp.backward(dy, gu)
    assert float((dx.double() - grad).norm()) <= 3 * ref.REL * float(grad.norm())
    assert torch.equal(y, mlp.forward(x, residual=x))
    _clean(gate_up, down)


def test_in_place_residual():
    lay, w = _linear("w4", 384, 208)
    for M in (1, 40, 300):
        x, res = _t(1, M, 384), _t(2, M, 208)
        want = lay.linear(x, residual=res)
        out = res.clone()
        assert lay.linear(x, residual=out, y=out) is out
        assert torch.equal(out, want)


@pytest.mark.parametrize("M", [1, 13, 40, 257])
def test_writes_nothing_else(M):
    """Guard rows around every output stay as they were."""
    K, N = 384, 208
    lay, _ = _linear("w4", K, N)
    gat, _, _ = _gated("w4", K, N)

    def guarded(*shape, dtype=torch.float16):
        n = int(np.prod(shape))
        buf = torch.full((n + 512,), 7.0, dtype=dtype, device=DEV)
        return buf, buf[256:256 + n].view(shape)

    (by, y), (bz, z), (bx, dx) = guarded(M, N), guarded(M, N), guarded(M, K)
    (bd, db), (bh, h), (bg, gu) = guarded(N, dtype=torch.float32), guarded(M, N), guarded(M, 2, N)
    (be, de) = guarded(2, N, dtype=torch.float32)
    x, dy = _t(1, M, K), _t(2, M, N)
    lay.linear(x, act="gelu", y=y, z=z)
    lay.linear_backward(dy, z=z, act="gelu", dx=dx, dbias=db)
    gat.forward(x, h=h, gu=gu)
    gat.backward(dy, gu, dx=dx, dbias=de)
    for buf, view in ((by, y), (bz, z), (bx, dx), (bd, db), (bh, h), (bg, gu), (be, de)):
        assert (buf[:256] == 7).all() and (buf[256 + view.numel():] == 7).all()


@pytest.mark.parametrize("M", [2, 16, 40, 300])
def test_non_finite_rows_stay_apart(M):
    """A row of infinities or NaN leaves the other rows' outputs as they are."""
    K, N = 384, 208
    lay, _ = _linear("w4", K, N)
    gat, _, _ = _gated("w4", K, N)
    x, dy = _t(1, M, K), _t(2, M, N)
    z, gu = _t(3, M, N), _t(4, M, 2, N)
    calls = [lambda a, d: lay.linear(a, act="silu"), lambda a, d: gat.forward(a),
             lambda a, d: lay.linear_backward(d, z=z, act="gelu"),
             lambda a, d: gat.backward(d, gu)]
    for call in calls:
        clean = call(x, dy)
        for bad in (float("inf"), float("nan")):
            xb, db = x.clone(), dy.clone()
            xb[M // 2], db[M // 2] = bad, bad
            out = call(xb, db)
            keep = [m for m in range(M) if m != M // 2]
            assert torch.equal(out[keep], clean[keep])
            assert not torch.isfinite(out[M // 2]).any()


def test_extreme_activations():
    """The largest fp16 inputs: no NaN from the activations' intermediate infinities."""
    K, N = 128, 16
    lay, w = _linear("w4", K, N)
    for M in (1, 20):
        x = torch.full((M, K), 0.0, dtype=torch.float16, device=DEV)
        x[:, 0] = 60000.0
        for act in ACTS:
            y, z = lay.linear(x, act=act), lay.linear(x)
            want = ref.act(act, z.double())
            assert torch.isfinite(y).all()
            assert torch.allclose(y.double(), want, rtol=2 * ref.U, atol=1e-6), act
        dy = torch.ones((M, N), dtype=torch.float16, device=DEV)
        for act in ACTS[1:]:
            for val in (60000.0, -60000.0):
                zz = torch.full((M, N), val, dtype=torch.float16, device=DEV)
                db = torch.empty(N, dtype=torch.float32, device=DEV)
                lay.linear_backward(dy, z=zz, act=act, dbias=db)
                assert torch.equal(db, torch.full_like(db, M if val > 0 else 0.0)), (act, val)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_reproducible(M):
    K, F = 2048, 592
    lay, _, _ = _gated("w4", K, F)
    x, dh = _t(1, M, K), _t(2, M, F)
    gu = _t(3, M, 2, F)
    first = None
    for _ in range(20):
        db = torch.empty((2, F), dtype=torch.float32, device=DEV)
        got = (lay.forward(x), lay.backward(dh, gu, dbias=db), db)
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    _clean(lay)


def test_one_workspace_for_different_layers():
    """Calls of other shapes, formats and entries in turn on one workspace."""
    big, _, _ = _gated("w4", 2048, 592)
    small, _ = _linear("w8", 384, 208)
    ws = max((big.new_workspace(300), small.new_workspace(300)), key=lambda t: t.numel())
    args = {M: (_t(M, M, 2048), _t(M + 1, M, 592), _t(M + 2, M, 2, 592), _t(M + 3, M, 384),
                _t(M + 4, M, 208), _t(M + 5, M, 208)) for M in (1, 9, 40, 300)}

    def calls(M, ws):
        x, dh, gu, x2, dy, z = args[M]
        db = torch.empty((2, 592), dtype=torch.float32, device=DEV)
        db2 = torch.empty(208, dtype=torch.float32, device=DEV)
        return [big.forward(x, workspace=ws), small.linear(x2, workspace=ws),
                big.backward(dh, gu, dbias=db, workspace=ws), db,
                small.linear_backward(dy, z=z, act="silu", dbias=db2, workspace=ws), db2]

    own = {M: calls(M, None) for M in args}
    for M in (300, 1, 40, 9, 1, 300, 9):
        assert all(torch.equal(a, b) for a, b in zip(own[M], calls(M, ws))), M
    assert ql.qlinear_read_error(ws) == 0


def test_streams():
    """Calls of one layer on two streams in turn, the inputs made on the call's stream."""
    lay, _, _ = _gated("w4", 2048, 592)
    for M in (1, 40, 300):
        x = _t(M, M, 2048)
        want = lay.forward(x)
        torch.cuda.synchronize()
        s = [torch.cuda.Stream(), torch.cuda.Stream()]
        outs = [lay.forward(x, stream=s[i % 2]) for i in range(8)]
        raw = lay.forward(x, stream=s[0].cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs + [raw])


def test_graphs():
    """Forward and backward captured and replayed with new inputs; two graphs with workspaces
    of their own replayed at the same time."""
    K, F = 2048, 640
    lay, _, _ = _gated("w4", K, F)
    down, _ = _linear("w8", F, K, seed=9)
    for M in (1, 40, 300):
        x, dy = _t(1, M, K), _t(2, M, K, std=0.25)
        gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV)
        graphs = []
        for _ in range(2):
            wa, wb = lay.new_workspace(M), down.new_workspace(M)
            xi, gi = x.clone(), gu.clone()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                h = lay.forward(xi, gu=gi, workspace=wa)
                y = down.linear(h, residual=xi, workspace=wb)
                dh = down.linear_backward(dy, workspace=wb)
                dx = lay.backward(dh, gi, workspace=wa)
            graphs.append((g, xi, y, dx, (wa, wb, h, dh, gi)))
        for seed in (5, 6):
            xn = _t(seed, M, K)
            h = lay.forward(xn, gu=gu)
            want_y = down.linear(h, residual=xn)
            want_dx = lay.backward(down.linear_backward(dy), gu)
            for _, xi, *_rest in graphs:
                xi.copy_(xn)
            torch.cuda.synchronize()
            streams = [torch.cuda.Stream(), torch.cuda.Stream()]
            for (g, *_rest), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            for _, _, y, dx, _keep in graphs:
                assert torch.equal(y, want_y) and torch.equal(dx, want_dx)
        del graphs


def test_capture_needs_a_reserved_workspace():
    lay, _ = _linear("w2", 384, 208, seed=30)
    x = _t(1, 40, 384)
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="reserve"):
        with torch.cuda.graph(g):
            lay.linear(x)
    lay.reserve(40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lay.linear(x)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, lay.linear(x))


def test_empty_batch():
    lay, _ = _linear("w4", 384, 208)
    gat, _, _ = _gated("w4", 384, 208)
    e = torch.empty
    f16 = dict(dtype=torch.float16, device=DEV)
    assert lay.linear(e((0, 384), **f16)).shape == (0, 208)
    assert gat.forward(e((0, 384), **f16)).shape == (0, 208)
    db = torch.ones(208, dtype=torch.float32, device=DEV)
    assert lay.linear_backward(e((0, 208), **f16), dbias=db).shape == (0, 384)
    assert (db == 0).all()
    assert gat.backward(e((0, 208), **f16), e((0, 2, 208), **f16)).shape == (0, 384)


def test_layer_refusals():
    lay, _ = _linear("w4", 384, 208)
    gat, _, _ = _gated("w4", 384, 208)
    x, res = _t(1, 4, 384), _t(2, 4, 208)
    with pytest.raises(ValueError, match="x must be"):
        lay.linear(x.float())
    with pytest.raises(ValueError, match="x must be"):
        lay.linear(_t(1, 384, 4).t())
    with pytest.raises(ValueError, match="on cpu"):
        lay.linear(x.cpu())
    with pytest.raises(ValueError, match="bias"):
        lay.linear(x, bias=res)
    with pytest.raises(ValueError, match="gu"):
        gat.backward(res, res)
    with pytest.raises(ql.QLinearError, match="NULL"):
        lay.linear_backward(res, act="silu")
    with pytest.raises(ql.QLinearError, match="UNSUPPORTED"):
        lay.linear(x, act="swish")
    with pytest.raises(ql.QLinearError, match="ALIAS"):
        lay.linear(x, y=res, z=res)
    sq, _ = _linear("w4", 384, 384)
    with pytest.raises(ql.QLinearError, match="ALIAS"):
        sq.linear(x, y=x)
    with pytest.raises(ql.QLinearError, match="WORKSPACE"):
        lay.linear(x, workspace=torch.zeros(1024, dtype=torch.uint8, device=DEV))
    for bad in ("w3", "outlier", "group"):
        if bad == "w3":
            l3 = layers.from_uniform(gen.uniform_layer(1, 384, 208, 3), DEV)
        elif bad == "outlier":
            l3 = layers.from_outlier(gen.outlier_layer(1, 384, 256), DEV)
        else:
            l3 = layers.from_uniform(gen.uniform_layer(1, 384, 208, 4, group=64), DEV)
        with pytest.raises(ValueError):
            l3.linear(x)


@pytest.mark.parametrize("M", [24, 64, 100, 200, 256, 520])
@pytest.mark.parametrize("fmt", FMTS)
def test_many_calls(fmt, M):
    """Thirty calls, each with dozens of units per pipeline (every code ring goes round many
    times, the decoding teams run apart), all bit-identical, in both directions, and right."""
    K, N = 4096, 2320
    lay, w = _linear(fmt, K, N, seed=50)
    x, dy = _t(M, M, K), _t(M + 1, M, N, std=0.25)
    y, dx = lay.linear(x), lay.linear_backward(dy)
    ref.check(y, ref.linear(x.double(), w)[0], "y")
    ref.check(dx, ref.linear_backward(dy.double(), None, w, "none")[0], "dx")
    for _ in range(30):
        assert torch.equal(lay.linear(x), y)
        assert torch.equal(lay.linear_backward(dy), dx)
    _clean(lay)


@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_two_calls_at_once(M):
    """Two layers' calls on two streams, overlapping as the device sees fit."""
    a, _, _ = _gated("w4", 2048, 592)
    b, _ = _linear("w8", 1024, 512)
    xa, xb = _t(1, M, 2048), _t(2, M, 1024)
    dh, gu, dy, z = _t(3, M, 592), _t(4, M, 2, 592), _t(5, M, 512), _t(6, M, 512)

    def call_a(**kw):
        return a.forward(xa, **kw), a.backward(dh, gu, **kw)

    def call_b(**kw):
        return b.linear(xb, act="gelu", **kw), b.linear_backward(dy, z=z, act="gelu", **kw)

    want = call_a() + call_b()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = [call_a(stream=s) + call_b(stream=t) for _ in range(20)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(u, v) for u, v in zip(g, want))
    _clean(a, b)


def test_more_rows_than_reserved():
    """Rows rise and fall; a policy table that changes the grid asks for a larger workspace."""
    lay, w = _linear("w4", 1024, 512, seed=60)
    for M in (1, 300, 8, 16, 700, 2):
        x = _t(M, M, 1024)
        ref.check(lay.linear(x), ref.linear(x.double(), w)[0], str(M))
    fresh, _ = _linear("w4", 1024, 512, seed=61)
    x = _t(1, 9, 1024)
    want = fresh.linear(x)
    ql.qlinear_policy_set([dict(fmt=4, N=512, K=1024, m_lo=1, m_hi=16, ctas=32)])
    try:
        assert torch.allclose(fresh.linear(x).float(), want.float(), rtol=2 ** -9, atol=2 ** -9)
    finally:
        ql.qlinear_policy_set([])
    _clean(lay, fresh)


def test_offsets_beyond_32_bits():
    """Outputs, kept values and gradients of more than 2^31 elements, checked at both ends."""
    K, N, M = 128, 65536, 33000
    assert M * N > 2 ** 31
    ends = [slice(0, 40), slice(M - 40, M)]
    x = _t(1, M, K)
    lay, w = _linear("w4", K, N)
    z = torch.empty((M, N), dtype=torch.float16, device=DEV)
    y = lay.linear(x, act="relu", z=z)
    for r in ends:
        wy, wz = ref.linear(x[r].double(), w, name="relu")
        ref.check(y[r], wy, "y")
        ref.check(z[r], wz, "z")
    dx = lay.linear_backward(y, z=z, act="silu")
    for r in ends:
        ref.check(dx[r], ref.linear_backward(y[r].double(), z[r].double(), w, "silu")[0], "dx")
    _clean(lay)
    del y, z, dx
    gat, wg, wu = _gated("w4", K, N // 2)
    gu = torch.empty((M, 2, N // 2), dtype=torch.float16, device=DEV)
    h = gat.forward(x, gu=gu)
    for r in ends:
        wh, wgu = ref.gated(x[r].double(), wg, wu)
        ref.check(h[r], wh, "h")
        ref.check(gu[r], wgu, "gu")
    h.clamp_(-1, 1)  # as a gradient: its product with the gate and up values stays in fp16
    dx = gat.backward(h, gu)
    for r in ends:
        want = ref.gated_backward(h[r].double(), gu[r].double(), wg, wu, "silu")[0]
        ref.check(dx[r], want, "dx")
    _clean(gat)
    lay._fused_ws = gat._fused_ws = ()  # gigabytes


def test_workspace_after_an_error_flag():
    """A flag in the workspace is reported once, and arrivals that a call left are cleared."""
    lay, _ = _linear("w4", 2048, 1168)
    x = _t(1, 40, 2048)
    want = lay.linear(x)
    ws = lay.new_workspace(40)
    words = ws.view(torch.int32)
    words[0] = 1
    words[64:96] = 1
    assert lay.fused_read_error(ws) == 1
    assert not ws.any() and lay.fused_read_error(ws) == 0
    assert torch.equal(lay.linear(x, workspace=ws), want)


def test_rising_lengths_keep_few_workspaces():
    """One buffer per doubling of the rows, not one per length; reserve() takes exactly the rows
    that it is given."""
    lay, _ = _linear("w4", 384, 208, seed=62)
    for M in range(1, 1025, 31):
        lay.linear_backward(_t(M, M, 208), z=_t(M, M, 208), act="silu")
    sizes = [w.numel() for w in lay._fused_ws]
    assert len(sizes) <= 11 and sizes == sorted(sizes)
    assert sizes[-1] == lay.new_workspace(1024).numel()
    assert sum(sizes[:-1]) <= 10 * sizes[-1]
    other, _ = _linear("w4", 384, 208, seed=63)
    other.reserve(1000)
    assert other._fused_ws[-1].numel() == other.new_workspace(1000).numel()


def test_one_workspace_for_a_model():
    """The largest layer's workspace serves every layer's calls, forward and backward."""
    lays = [_linear("w4", 2048, 1168)[0], _linear("w8", 384, 208)[0], _gated("w4", 384, 208)[0]]
    M = 300
    ws = max((lay.new_workspace(M) for lay in lays), key=lambda t: t.numel())
    x, x2 = _t(1, M, 2048), _t(2, M, 384)
    z, dy, z2, dy2, gu = (_t(3, M, 1168), _t(4, M, 1168), _t(5, M, 208), _t(6, M, 208),
                          _t(7, M, 2, 208))

    def step(w):
        return [lays[0].linear(x, workspace=w), lays[1].linear(x2, act="gelu", workspace=w),
                lays[2].forward(x2, workspace=w),
                lays[2].backward(dy2, gu, workspace=w),
                lays[1].linear_backward(dy2, z=z2, act="gelu", workspace=w),
                lays[0].linear_backward(dy, z=z, act="silu", workspace=w)]

    assert all(torch.equal(a, b) for a, b in zip(step(None), step(ws)))
    assert ql.qlinear_read_error(ws) == 0


def test_growth_falls_back_to_the_rows_asked_for(monkeypatch):
    """Where the next power of two of rows does not fit into memory."""
    lay, w = _linear("w4", 384, 208, seed=66)
    new = lay.new_workspace

    def small(rows, backward=True):
        if rows > 300:
            raise torch.OutOfMemoryError("no room")
        return new(rows, backward)

    monkeypatch.setattr(lay, "new_workspace", small)
    x = _t(1, 300, 384)
    ref.check(lay.linear(x), ref.linear(x.double(), w)[0], "y")
    assert len(lay._fused_ws) == 1


def test_error_flags_of_outgrown_workspaces():
    """A flag in a buffer that the layer has outgrown (a captured graph may use it) is reported,
    and the arrivals beside it are cleared."""
    lay, _ = _linear("w4", 2048, 1168, seed=64)
    x = _t(1, 40, 2048)
    lay.reserve(40)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lay.linear(x)
    old = lay._fused_ws[-1]
    lay.reserve(300)
    assert lay._fused_ws[-1] is not old
    g.replay()
    torch.cuda.synchronize()
    want = y.clone()
    words = old.view(torch.int32)
    words[0] = 2
    words[64:96] = 1
    assert lay.fused_read_error() == 2
    assert not old[256:16384].any() and lay.fused_read_error() == 0
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_error_flags_wait_for_other_streams():
    """The flags are those of every call that was made, also of one that still runs on a stream
    that nobody waited for."""
    lay, _ = _linear("w4", 1024, 1168, seed=65)
    x = _t(1, 20, 1024)
    lay.linear(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ql.qlinear_debug_wait_test(2000, 20000, 0)
    try:
        lay.linear(x, stream=s)  # gives up after 2 ms, done after 20
    finally:
        ql.qlinear_debug_wait_test()
    assert lay.fused_read_error() != 0
    assert lay.fused_read_error() == 0


def test_tensors_that_require_a_gradient_are_refused():
    """Autograd would drop the gradient silently; inside an autograd.Function, or under no_grad,
    the calls run."""
    lay, w = _linear("w4", 384, 208)
    gat, _, _ = _gated("w4", 384, 208)
    x, dy = _t(1, 4, 384), _t(2, 4, 208)
    gu = _t(3, 4, 2, 208)
    want = lay.linear(x)
    for bad in (x, dy, gu):
        bad.requires_grad_(True)
    for call in (lambda: lay.linear(x), lambda: lay.linear(x.detach(), residual=dy),
                 lambda: lay.linear(x * 1), lambda: gat.forward(x),
                 lambda: lay.linear_backward(dy), lambda: gat.backward(dy.detach(), gu)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
    with torch.no_grad():
        assert torch.equal(lay.linear(x), want)
        assert torch.equal(gat.backward(dy, gu), gat.backward(dy.detach(), gu.detach()))

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return lay.linear(x)

        @staticmethod
        def backward(ctx, dy):
            return lay.linear_backward(dy.contiguous())

    y = Linear.apply(x)
    assert torch.equal(y, want)
    y.backward(dy.detach())
    ref.check(x.grad, ref.linear_backward(dy.detach().double(), None, w, "none")[0], "dx")


@pytest.mark.parametrize("M", [1, 33, 260])
def test_feed_forward_block_with_biases(M):
    """Biases, their gradients, outputs of the caller's and one workspace for the whole block."""
    K, F = 512, 1152
    gate_up, wg, wu = _gated("w4", K, F)
    down, wd = _linear("w8", F, K, seed=9)
    mlp = layers.GatedMLP(gate_up, down)
    ws = mlp.new_workspace(M)
    x, dy = _t(1, M, K), _t(2, M, K, std=0.25)
    bias, down_bias = _t(3, 2, F, std=0.3), _t(4, K, std=0.3)
    gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    db = torch.empty((2, F), dtype=torch.float32, device=DEV)
    ddb = torch.empty(K, dtype=torch.float32, device=DEV)
    assert mlp.forward(x, residual=x, gu=gu, bias=bias, down_bias=down_bias, y=y,
                       workspace=ws) is y
    assert mlp.backward(dy, gu, dx=dx, dbias=db, ddown_bias=ddb, workspace=ws) is dx
    xd, bd, dd = (t.double().requires_grad_(True) for t in (x, bias, down_bias))
    want = (ref.act("silu", xd @ wg + bd[0]) * (xd @ wu + bd[1])) @ wd + dd + x.double()
    grads = torch.autograd.grad(want, (xd, bd, dd), dy.double())
    for got, exp in ((y, want.detach()), (dx, grads[0]), (db, grads[1]), (ddb, grads[2])):
        assert float((got.double() - exp).norm()) <= 3 * ref.REL * float(exp.norm())
    assert ql.qlinear_read_error(ws) == 0


def test_feed_forward_blocks_replayed_at_once():
    """Two graphs of one block, each with a workspace of its own, replayed at the same time."""
    M, K, F = 100, 512, 1152
    mlp = layers.GatedMLP(_gated("w4", K, F)[0], _linear("w8", F, K, seed=9)[0])
    x, dy = _t(1, M, K), _t(2, M, K, std=0.25)
    gu = torch.empty((M, 2, F), dtype=torch.float16, device=DEV)
    want_y, want_dx = mlp.forward(x, gu=gu), mlp.backward(dy, gu)
    graphs = []
    for _ in range(2):
        ws, g = mlp.new_workspace(M), torch.cuda.CUDAGraph()
        kept = torch.empty_like(gu)
        with torch.cuda.graph(g):
            y = mlp.forward(x, gu=kept, workspace=ws)
            dx = mlp.backward(dy, kept, workspace=ws)
        graphs.append((g, y, dx, ws, kept))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for (g, y, dx, *_), s in zip(graphs, streams):
            y.zero_(), dx.zero_()
        torch.cuda.synchronize()
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, y, dx, *_ in graphs:
            assert torch.equal(y, want_y) and torch.equal(dx, want_dx)


@pytest.mark.parametrize("M", [1, 9, 40])
def test_shapes_beyond_the_gemv(M, monkeypatch):
    """More units times CTAs than the GEMV's 32-bit counts hold (a grid capped at its units gets
    there with a small layer): the tensor-core product takes over, at any M."""
    K, N = 92800, 8192  # 725 x 64 units
    monkeypatch.setenv("QLINEAR_MAX_CTAS", "1000000")
    rows = 64
    assert (K // 128) * (N // 128) * min(1000000, (K // 128) * (N // 128)) >= 2 ** 31
    nbytes = ql.qlinear_fused_workspace_bytes(2, rows, N, K, False)
    assert nbytes > 0
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=DEV)
    q = torch.full((K * N // 4,), 0b01010101, dtype=torch.uint8, device=DEV)  # every code 1
    p0 = torch.full((K // 128 * N,), 0.5, dtype=torch.float16, device=DEV)
    p1 = torch.zeros(K // 128 * N, dtype=torch.float16, device=DEV)
    x = torch.zeros((M, K), dtype=torch.float16, device=DEV)
    x[:, ::29] = torch.arange(1, M + 1, device=DEV).half().unsqueeze(1) / 64
    y = torch.empty((M, N), dtype=torch.float16, device=DEV)
    ql.qlinear_linear(2, x, q, p0, p1, y, M, N, K, ws)
    assert torch.equal(y, (x.double().sum(1) / 2).half().unsqueeze(1).expand(M, N))
    h = torch.empty((M, N // 2), dtype=torch.float16, device=DEV)
    ql.qlinear_gated(2, x / 64, q, p0, p1, h, M, N // 2, K, ws, act="relu")
    want = (x.double().sum(1) / 128) ** 2
    assert torch.equal(h, want.half().unsqueeze(1).expand(M, N // 2))
    assert ql.qlinear_read_error(ws) == 0
