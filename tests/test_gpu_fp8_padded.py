"""Rows of no expert: a buffer of fixed capacity of which the experts' rows fill a part, through the
block and the norm's backward pass on the GPU.  Such rows have no gradient from the products."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import fp8_ref as ref
    from weight_only_quantized_gemv_b200 import layers

TYPES = [torch.float16, torch.bfloat16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _nan_filled(make):
    """Tensors made with every byte set: NaN in each of the types."""
    def made(*args, **kw):
        t = make(*args, **kw)
        t.view(torch.uint8).fill_(255)
        return t
    return made


def _randn(gen, *shape, dtype, std=0.1):
    return (std * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def _experts_block(gen, E, H, F, dtype):
    mats = [layers.Fp8Experts(*layers.fp8_quantize_weights(_randn(gen, E, *shape, dtype=dtype,
                                                                  std=0.05)))
            for shape in ((2 * F, H), (H, F))]
    weight = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
    return layers.Fp8GatedMLP(*mats, layers.RMSNorm(weight))


def _offsets(front, rows, E, rng):
    at = [front + a for a in ref.split(rows, E, rng)]
    at[-1] = front + rows
    return torch.tensor(at, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,H,F,front,rows,behind", [
    (4, 256, 144, 3, 32, 5), (3, 1040, 384, 100, 563, 37), (2, 512, 128, 0, 1, 400),
    (2, 512, 128, 400, 1, 0), (5, 256, 128, 30, 0, 20)])
def test_block_backward(E, H, F, front, rows, behind, dtype, monkeypatch):
    gen, M = _gen(H + rows), front + rows + behind
    block = _experts_block(gen, E, H, F, dtype)
    at, own = _offsets(front, rows, E, random.Random(rows)), slice(front, front + rows)
    monkeypatch.setattr(layers, "_new", _nan_filled(layers._new))
    monkeypatch.setattr(layers.RMSNorm, "_fused_new",
                        staticmethod(_nan_filled(layers.RMSNorm._fused_new)))
    x, r = (ref.activations(gen, M, H, dtype) for _ in range(2))
    x[:front], x[front + rows:] = float("inf"), float("nan")
    total, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    gu = torch.full((M, 2 * F), float("nan"), dtype=dtype, device="cuda")
    y = block.forward(x, r, at, total=total, rstd=rstd, gu=gu)
    assert bool(torch.isfinite(y[own]).all()) and bool(torch.isfinite(gu[own]).all())
    dy, dt = _randn(gen, M, H, dtype=dtype), _randn(gen, M, H, dtype=dtype)
    dy[:front], dy[front + rows:] = float("nan"), float("inf")

    q, s = layers.fp8_quantize(dy)
    dh = block.down.backward(q, s, at, dtype=dtype)
    q, s = layers.fp8_gated_backward(dh, gu, "silu")
    dv = block.gate_up.backward(q, s, at, dtype=dtype)
    for through in (None, dt):
        dweight = torch.full((H,), float("nan"), device="cuda")
        kept = None if through is None else through.clone()
        dx = block.backward(dy, gu, total, rstd, at, dtotal=kept, dweight=dweight)
        want, err, want_w, err_w = ref.norm_backward(
            dv[own], total[own], rstd[own], block.norm.weight,
            None if through is None else through[own])
        ref.check(dx[own], want, err, "dx")
        assert bool(((dweight.double() - want_w).abs() <= err_w).all())
        none = torch.zeros_like(dx) if through is None else through
        for rest in (slice(0, front), slice(front + rows, M)):
            assert torch.equal(dx[rest], none[rest])
        if through is not None:  # in place
            again = block.backward(dy, gu, total, rstd, at, dtotal=kept, dx=kept)
            assert again is kept and torch.equal(kept, dx)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("through", [False, True])
@pytest.mark.parametrize("M,K", [(1, 16), (9, 144), (601, 1024), (700, 2064), (301, 8208),
                                 (300, 14336), (5, 16400), (160, 32768)])
def test_norm_backward(M, K, through, dtype):
    gen, rng = _gen(M + K), random.Random(M)
    t, dy = ref.activations(gen, M, K, dtype), _randn(gen, M, K, dtype=dtype)
    weight = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dtype)
    dt = _randn(gen, M, K, dtype=dtype) if through else None
    norm = layers.RMSNorm(weight)
    rstd = torch.empty(M, device="cuda")
    norm.forward(t, rstd=rstd)
    ends = [(0, M), (0, 0), (M, M), (M // 3, M - M // 4), (M // 2, M // 2 + 1), (-5, M + 7),
            (M + 3, M + 9), (M // 2, M // 3 - 1)]
    for lo, hi in ends:
        a, b = min(max(lo, 0), M), min(max(hi, 0), M)
        b = max(a, b)
        middle = sorted(rng.randint(a, b) for _ in range(rng.randint(0, 3)))
        at = torch.tensor([lo, *middle, hi], dtype=torch.int32, device="cuda")
        part = dy.clone()
        part[:a], part[b:] = float("nan"), float("inf")
        dweight = torch.full((K,), float("nan"), device="cuda")
        dx = norm.backward(part, t, rstd, dtotal=dt, dweight=dweight, offsets=at)
        alone = norm.backward(part, t, rstd, dtotal=dt, offsets=at)
        assert torch.equal(alone, dx)
        none = torch.zeros_like(dx) if dt is None else dt
        assert torch.equal(dx[:a], none[:a]) and torch.equal(dx[b:], none[b:])
        if b > a:  # a row's values do not go by the others
            rows = norm.backward(dy[a:b], t[a:b], rstd[a:b], dtotal=None if dt is None else dt[a:b])
            assert torch.equal(dx[a:b], rows)
        _, _, want, err = ref.norm_backward(dy[a:b], t[a:b], rstd[a:b], weight)
        assert bool(((dweight.double() - want).abs() <= err).all())
    full = torch.empty(K, device="cuda")
    norm.backward(dy, t, rstd, dweight=full)
    again = torch.empty(K, device="cuda")
    norm.backward(dy, t, rstd, dweight=again, offsets=torch.tensor([0, M], dtype=torch.int32,
                                                                  device="cuda"))
    assert torch.equal(again, full)


def test_a_graph_takes_new_offsets():
    """One graph of the block's both directions, replayed for other fillings of its rows."""
    E, H, F, M, dtype = 4, 512, 256, 200, torch.bfloat16
    gen = _gen(1)
    block = _experts_block(gen, E, H, F, dtype)
    x, r = (ref.activations(gen, M, H, dtype) for _ in range(2))
    dy, dt = _randn(gen, M, H, dtype=dtype), _randn(gen, M, H, dtype=dtype)
    total, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
    gu = torch.full((M, 2 * F), float("nan"), dtype=dtype, device="cuda")
    dweight = torch.empty(H, device="cuda")
    at = torch.zeros(E + 1, dtype=torch.int32, device="cuda")

    def run():
        block.forward(x, r, at, total=total, rstd=rstd, gu=gu)
        return block.backward(dy, gu, total, rstd, at, dtotal=dt, dweight=dweight)

    block.reserve(M)
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for front, rows in ((0, M), (10, 60), (150, 50), (7, 0), (0, 1)):
        at.copy_(_offsets(front, rows, E, random.Random(rows)))
        want = [t.clone() for t in (run(), dweight)]
        dweight.fill_(float("nan"))
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(dweight, want[1])
        assert bool(torch.isfinite(dweight).all()) and (rows or not dweight.any())
        assert torch.equal(out[:front], dt[:front])
    del graph


def test_offsets_of_the_norm_are_checked():
    K, M = 256, 8
    norm = layers.RMSNorm(torch.ones(K, dtype=torch.float16, device="cuda"))
    x, rstd = torch.randn(M, K, device="cuda").half(), torch.ones(M, device="cuda")
    for at in (torch.zeros(3, dtype=torch.int64, device="cuda"), torch.zeros(3, dtype=torch.int32),
               torch.zeros(1, dtype=torch.int32, device="cuda"),
               torch.zeros(1026, dtype=torch.int32, device="cuda"),
               torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
               torch.zeros(6, dtype=torch.int32, device="cuda")[::2]):
        with pytest.raises(ValueError):
            norm.backward(x, x, rstd, offsets=at)
