"""The 8-bit floating-point layers under graphs, streams, threads, shared workspaces, bounded waits
and sizes beyond 32 bits, on the GPU."""
import copy
import random
import threading

import pytest

from synth import gen as synth_gen

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from tests import fp8_ref as ref
    from weight_only_quantized_gemv_b200 import layers

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)
    yield
    ql.qlinear_debug_wait_test()  # defaults again, whatever the test did


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(gen, M, C):
    return ref.quantize(torch.randn(M, C, generator=gen, device="cuda").double())


def _same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------------------
# bounded waits


@pytest.mark.parametrize("late", ["copy", "mma"])
@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("N,K", [(1024, 1168), (1152, 18944)])
@pytest.mark.parametrize("M", [5, 20, 60, 300])
def test_product_gives_up(M, N, K, backward, late):
    gen = _gen(M + N)
    lay = layers.Fp8Linear(*ref.weights(gen, N, K))
    q, s = _codes(gen, M, N if backward else K)
    call = lay.backward if backward else lay.forward
    want = call(q, s)
    assert lay.fused_read_error() == 0
    ql.qlinear_debug_wait_test(2000, 10000 if late == "copy" else 0, 10000 if late == "mma" else 0)
    call(q, s)
    torch.cuda.synchronize()
    assert lay.fused_read_error(), "the late step was not reported"
    ql.qlinear_debug_wait_test()
    for _ in range(3):
        assert torch.equal(call(q, s), want)
    assert lay.fused_read_error() == 0


@pytest.mark.parametrize("M", [3, 40, 200])
def test_no_flag_behind_a_long_kernel(M):
    """The limit of a call's waits begins once the kernels before it have ended."""
    gen = _gen(M)
    lay = layers.Fp8Linear(*ref.weights(gen, 2320, 2048))
    small = layers.Fp8Linear(*ref.weights(gen, 16, 128))
    q, s = _codes(gen, M, 2048)
    qs, ss = _codes(gen, 20, 128)
    want, first = lay.forward(q, s), small.forward(qs, ss)
    ql.qlinear_debug_wait_test(1000000, 60000, 0)  # one CTA, for 60 ms
    out = small.forward(qs, ss)
    ql.qlinear_debug_wait_test(5000, 0, 0)
    got = lay.forward(q, s)
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(got, want)
    assert lay.fused_read_error() == 0 and small.fused_read_error() == 0


# ---------------------------------------------------------------------------
# streams, threads, graphs


def _block(gen, E, H, F, dtype=torch.bfloat16):
    lead = (E,) if E else ()
    kind = layers.Fp8Experts if E else layers.Fp8Linear
    mats = [kind(*layers.fp8_quantize_weights(
        (torch.randn(*lead, *shape, generator=gen, device="cuda") * 0.05).to(dtype)))
        for shape in ((2 * F, H), (H, F))]
    weight = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
    return layers.Fp8GatedMLP(*mats, layers.RMSNorm(weight))


class _Case:
    """A block's inputs and everything that a forward and a backward call give."""

    def __init__(self, block, gen, M, E):
        H, F = block.gate_up.K, block.down.K
        self.x, self.r = (ref.activations(gen, M, H, torch.bfloat16) for _ in range(2))
        self.dy = (0.1 * torch.randn(M, H, generator=gen, device="cuda")).bfloat16()
        self.at = (torch.tensor(ref.split(M, E, random.Random(M)), dtype=torch.int32,
                                device="cuda") if E else None)
        self.total, self.gu = torch.empty_like(self.x), self.x.new_empty(M, 2 * F)
        self.rstd = torch.empty(M, device="cuda")
        self.dweight = torch.empty(H, device="cuda")

    def run(self, block, workspace=None, stream=None):
        # (rows of no expert keep what the outputs were made with: nothing here)
        y = block.forward(self.x, self.r, self.at, total=self.total, rstd=self.rstd, gu=self.gu,
                          workspace=workspace, stream=stream)
        dx = block.backward(self.dy, self.gu, self.total, self.rstd, self.at,
                            dweight=self.dweight, workspace=workspace, stream=stream)
        return [y, dx, self.dweight, self.total, self.gu]


def _rows_of_experts(case, outs):
    if case.at is None:
        return [o.clone() for o in outs]
    n = int(case.at[-1])
    return [o.clone() if o.dim() == 1 else o[:n].clone() for o in outs]


@pytest.mark.parametrize("E", [0, 4])
@pytest.mark.parametrize("M", [1, 50, 300])
def test_graphs(M, E):
    """Two graphs of one block, each with a workspace of its own, replayed at the same time with
    new inputs."""
    block = _block(_gen(M), E, 512, 384)
    block.reserve(M)
    cases = [_Case(block, _gen(10 + i), M, E) for i in range(2)]
    for c in cases:
        c.run(block)
    graphs = []
    for c in cases:
        ws = block.new_workspace(M)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = c.run(block, workspace=ws)
        graphs.append((g, outs, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for k in range(3):
        fresh = [_Case(block, _gen(20 + 2 * k + i), M, E) for i in range(2)]
        want = [_rows_of_experts(f, f.run(block)) for f in fresh]
        for c, f in zip(cases, fresh):
            for name in ("x", "r", "dy"):
                getattr(c, name).copy_(getattr(f, name))
        torch.cuda.synchronize()
        for _ in range(4):
            for (g, *_rest), st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for c, (_, outs, ws), w in zip(cases, graphs, want):
            for a, b in zip(_rows_of_experts(c, outs), w):
                assert torch.equal(a, b)
            assert ql.qlinear_read_error(ws) == 0
    del graphs


def test_capture_needs_a_reserved_workspace():
    lay = layers.Fp8Linear(*ref.weights(_gen(1), 256, 256))
    q, s = _codes(_gen(2), 4, 256)
    with pytest.raises(RuntimeError, match="reserve"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            lay.forward(q, s)
    lay.reserve(4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lay.forward(q, s)
    g.replay()
    assert torch.equal(y, lay.forward(q, s))


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("streams", [1, 4])
def test_threads_get_their_own_results(M, streams):
    block = _block(_gen(3), 0, 512, 384)
    block.reserve(M)
    cases = [_Case(block, _gen(30 + i), M, 0) for i in range(4)]
    want = [[o.clone() for o in c.run(block)] for c in cases]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(streams)]
    errors = []

    def caller(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(st[i % streams]):
                for _ in range(15):
                    outs = cases[i].run(block, stream=st[i % streams])
                    assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i
        except BaseException as e:  # noqa: BLE001 - reported below
            errors.append(e)

    ts = [threading.Thread(target=caller, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    if errors:
        raise errors[0]
    assert block.gate_up.fused_read_error() == block.down.fused_read_error() == 0


def test_outputs_are_made_on_the_calls_stream():
    """Calls with a stream given, from another current one: results as without, used there."""
    lay = layers.Fp8Linear(*ref.weights(_gen(4), 512, 512))
    x = ref.activations(_gen(5), 64, 512, torch.float16)
    q, s = layers.fp8_quantize(x)
    want = lay.forward(q, s)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (st, st.cuda_stream):
        for _ in range(20):
            q2, s2 = layers.fp8_quantize(x, stream=stream)
            y = lay.forward(q2, s2, stream=stream)
            st.synchronize()
            assert _same(q2, q) and torch.equal(s2, s) and torch.equal(y, want)


def test_a_copied_layer_has_a_lock_and_workspaces_of_its_own():
    lay = layers.Fp8Linear(*ref.weights(_gen(6), 256, 384))
    norm = layers.RMSNorm(torch.ones(256, dtype=torch.float16, device=DEV))
    q, s = _codes(_gen(7), 4, 384)
    want = lay.forward(q, s)
    for other in (copy.deepcopy(lay), copy.copy(lay)):
        assert other._fused_lock is not lay._fused_lock and not other._fused_ws
        assert torch.equal(other.forward(q, s), want)
    assert copy.deepcopy(norm)._fused_lock is not norm._fused_lock


def test_one_workspace_serves_the_fused_layers_too():
    """Calls of W4 and e4m3 layers and of the norm in turn with one workspace."""
    K, N, M = 1024, 1040, 300
    w4 = layers.from_uniform(synth_gen.uniform_layer(5, K, N, 4), DEV)
    f8 = layers.Fp8Linear(*ref.weights(_gen(8), N, K))
    norm = layers.RMSNorm(torch.ones(K, dtype=torch.float16, device=DEV))
    ws = max((lay.new_workspace(M) for lay in (w4, f8, norm)), key=lambda t: t.numel())
    dw, rstd = torch.empty(K, device=DEV), torch.rand(M, device=DEV)
    first = {}
    for turn in range(3):
        for m in (1, 12, 30, 100, M):
            x = ref.activations(_gen(m), m, K, torch.float16)
            q, s = layers.fp8_quantize(x)
            got = [w4.linear(x, workspace=ws), f8.forward(q, s, workspace=ws),
                   norm.backward(x, x, rstd[:m], dweight=dw, workspace=ws), dw.clone(),
                   w4.linear_backward(w4.linear(x, workspace=ws), act="none", workspace=ws)]
            want = first.setdefault(m, [t.clone() for t in got])
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (turn, m)
    want, err = ref.product(q, s, f8.codes, f8.scales)
    ref.check(first[M][1], want, err)
    assert ql.qlinear_read_error(ws) == 0


# ---------------------------------------------------------------------------
# sizes


def test_rows_and_outputs_beyond_32_bits():
    """More than 2^31 elements of x, codes and y; rows at the far end are right."""
    M, K, N = 132000, 16384, 16
    x = torch.zeros(M, K, dtype=torch.float16, device=DEV)
    last = ref.activations(_gen(9), 300, K, torch.float16)
    x[-300:] = last
    q, s = layers.fp8_quantize(x)
    assert q.numel() > 2 ** 31
    ref.check_codes(q[-300:], s[-300:], last.double())
    assert not q[:1000].view(torch.uint8).any()
    lay = layers.Fp8Linear(*ref.weights(_gen(10), N, K))
    y = lay.forward(q, s)
    want, err = ref.product(q[-300:], s[-300:], lay.codes, lay.scales)
    ref.check(y[-300:], want, err)
    del x, y
    # ... and of the backward product's output
    dq, ds = _codes(_gen(11), 300, N)
    q2 = torch.zeros(M, N, dtype=torch.float8_e4m3fn, device=DEV)
    s2 = torch.ones(M, 1, device=DEV)
    q2[-300:], s2[-300:] = dq, ds
    dx = lay.backward(q2, s2)
    assert dx.numel() > 2 ** 31
    want, err = ref.product(dq, ds, lay.codes, lay.scales, True)
    ref.check(dx[-300:], want, err)
    assert not dx[:1000].any() and lay.fused_read_error() == 0


def test_weights_beyond_32_bits():
    """Experts whose matrices together pass 2^31 codes: the last one's rows are right."""
    E, N, K = 40, 8192, 8192
    codes = torch.zeros(E, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.ones(E, N // 128, K // 128, device=DEV)
    c, s = ref.weights(_gen(12), N, K)
    codes[-1], scales[-1] = c, s
    lay = layers.Fp8Experts(codes, scales)
    at = torch.tensor([0] * E + [9], dtype=torch.int32, device=DEV)
    for backward in (False, True):
        q, qs = _codes(_gen(13), 9, K)
        out = (lay.backward if backward else lay.forward)(q, qs, at)
        want, err = ref.product(q, qs, c, s, backward)
        ref.check(out, want, err)


@pytest.mark.parametrize("seed", range(6))
def test_random_shapes(seed):
    """Shapes, splits, types and directions by chance, several calls on one layer."""
    rng, gen = random.Random(seed), _gen(100 + seed)
    for _ in range(6):
        E = rng.choice([1, 2, 5, 17, 64])
        N, K = 16 * rng.randint(1, 70), 16 * rng.randint(1, 70)
        lay = layers.Fp8Experts(*ref.weights(gen, E, N, K))
        for _ in range(3):
            backward = rng.random() < 0.5
            M = int(2 ** rng.uniform(0, 11))
            at = torch.tensor(ref.split(M, E, rng, rng.choice([0.0, 0.3, 0.8])),
                              dtype=torch.int32, device=DEV)
            q, s = _codes(gen, M, N if backward else K)
            out = torch.zeros(M, K if backward else N, device=DEV,
                              dtype=rng.choice([torch.float16, torch.bfloat16]))
            (lay.backward if backward else lay.forward)(q, s, at, out)
            for a, b, want, err in ref.grouped(q, s, at, lay.codes, lay.scales, backward):
                ref.check(out[a:b], want, err, f"E={E} N={N} K={K} M={M} {backward}")
            assert not out[int(at[-1]):].any()
        assert lay.fused_read_error() == 0


# ---------------------------------------------------------------------------
# a norm's weight that the stream's work just before the call writes


@pytest.mark.parametrize("writer", ["product", "step"])
@pytest.mark.parametrize("M,K", [(1, 256), (3, 4096), (700, 1040)])
def test_norm_weight_in_stream_order(M, K, writer):
    gen = _gen(M + K)
    lin = layers.Fp8Linear(*ref.weights(gen, K, 16384))
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    rstd = torch.rand(M, generator=gen, device="cuda") + 0.5
    norm = layers.RMSNorm(torch.zeros(K, dtype=torch.bfloat16, device="cuda"))
    inputs = [_codes(gen, 1, 16384) for _ in range(6)]

    def write(i, w):
        if writer == "product":  # lets the next grid start before it has written
            lin.forward(*inputs[i], y=w.view(1, K))
        else:
            for _ in range(4):
                w.add_(i + 1.0)

    def run(wait):
        norm.weight.zero_()
        got = []
        for i in range(len(inputs)):
            for backward in (False, True):
                write(i, norm.weight)
                if wait:
                    torch.cuda.synchronize()
                dw = torch.empty(K, device="cuda")
                got += ([norm.backward(dy, x, rstd, dweight=dw), dw] if backward
                        else norm.forward(x))
        torch.cuda.synchronize()
        return got

    want = run(True)
    assert not _same(want[1], want[5])  # the weight matters (the codes' scales)
    for a, b in zip(run(False), want, strict=True):
        assert _same(a, b)


# ---------------------------------------------------------------------------
# a norm's weight gradient from a set of sums per multiprocessor, joined by blocks of either size


@pytest.mark.parametrize("K", [9472, 9488, 14336])
@pytest.mark.parametrize("M", [147, 148, 149, 300])
def test_norm_weight_sums_of_wide_rows(M, K):
    gen = _gen(M + K)
    t = ref.activations(gen, M, K, torch.bfloat16)
    weight = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).bfloat16()
    dy = (0.1 * torch.randn(M, K, generator=gen, device="cuda")).bfloat16()
    norm = layers.RMSNorm(weight, eps=1e-6)
    rstd = torch.empty(M, device="cuda")
    norm.forward(t, rstd=rstd)
    dweight = torch.full((K,), float("nan"), device="cuda")
    dx = norm.backward(dy, t, rstd, dweight=dweight)
    want, err, want_w, err_w = ref.norm_backward(dy, t, rstd, weight, None)
    ref.check(dx, want, err, "dx")
    off = (dweight.double() - want_w).abs()
    assert bool((off <= err_w).all()), (off / err_w).max().item()
