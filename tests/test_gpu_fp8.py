"""The 8-bit floating-point layers on the GPU against fp64 (tests/fp8_ref.py derives the bounds)."""
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from tests import fp8_ref as ref
    from weight_only_quantized_gemv_b200 import layers

TYPES = [torch.float16, torch.bfloat16]
F8 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _empty(*shape, dtype=torch.float32):
    """Uninitialised memory that shows: every byte set."""
    return torch.full(shape, 0, dtype=dtype, device="cuda").view(torch.uint8).fill_(255).view(dtype)


# ---------------------------------------------------------------------------
# rows


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (3, 128), (2, 144), (5, 272), (7, 4096), (64, 2064),
                                 (300, 8192), (2, 18448)])
def test_quantize(M, K, dtype):
    x = ref.activations(_gen(M + K), M, K, dtype)
    q, s = layers.fp8_quantize(x, q=_empty(M, K, dtype=F8),
                               scales=_empty(M, ref.blocks(K)))
    ref.check_codes(q, s, x.double(), what=f"{M}x{K}")


def test_quantize_of_strided_rows_zeros_and_tiny_values():
    x = ref.activations(_gen(1), 9, 512, torch.bfloat16)
    x[2, 128:256] = 0
    x[3, 256:384] = 2.0 ** -120       # below the floor: codes of zero
    x[4, :128] *= 2.0 ** -60
    x[5, 7] = -3e38
    part = x[::2, 64:480]
    assert not part.is_contiguous()
    q, s = layers.fp8_quantize(part)
    ref.check_codes(q, s, part.double())
    assert (s[1, 1:2] > 0).all()
    one = x[4:5, 64:480]              # one row: its stride says nothing
    q1, s1 = layers.fp8_quantize(one)
    assert torch.equal(q1.view(torch.uint8), q[2:3].view(torch.uint8)) and torch.equal(s1, s[2:3])


def test_quantize_shows_nan_and_infinity():
    x = torch.ones(3, 384, dtype=torch.float16, device="cuda")
    x[0, 5], x[1, 200], x[2, 383] = float("nan"), float("inf"), -float("inf")
    q, s = layers.fp8_quantize(x)
    bad = torch.tensor([[1, 0, 0], [0, 1, 0], [0, 0, 1]], device="cuda", dtype=torch.bool)
    assert torch.equal(~torch.isfinite(s), bad)
    assert torch.isnan(q.float()[[0, 1, 2], [5, 200, 383]]).all()
    values = q.float() * ref.spread(s, 384).float()
    assert torch.equal(torch.isnan(values).view(3, 3, 128).any(2), bad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(16, 16), (128, 128), (400, 272), (2, 144, 528)])
def test_quantize_weights(shape, dtype):
    w = (torch.randn(*shape, generator=_gen(4), device="cuda") * 0.02).to(dtype)
    w.view(-1, shape[-1])[0, :7] = 0
    codes, scales = layers.fp8_quantize_weights(w)
    N, K = shape[-2:]
    full = ref.spread2(scales, N, K)
    pad = torch.nn.functional.pad(w.double(), (0, -K % 128, 0, -N % 128))
    top = pad.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128)).abs().amax((-3, -1))
    want = top.clamp_min(ref.FLOOR) / ref.TOP
    assert ((scales.double() - want).abs() <= 2.0 ** -23 * want).all()
    x = w.double() / full
    off = (codes.double() - x.clamp(-ref.TOP, ref.TOP)).abs()
    assert (off <= ref.half_step(x.clamp(-ref.TOP, ref.TOP)) + x.abs() * 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,residual", [(1, 16, True), (1, 4096, True), (4, 144, False),
                                          (3, 8192, True), (130, 2064, True), (2, 8208, False),
                                          (5, 16384, True), (2, 32768, True), (700, 1040, False)])
def test_norm(M, K, residual, dtype):
    gen = _gen(M * K)
    x = ref.activations(gen, M, K, dtype)
    r = ref.activations(gen, M, K, dtype, 2.0) if residual else None
    weight = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dtype)
    layer = layers.RMSNorm(weight, eps=1e-5)
    total, y, rstd = _empty(M, K, dtype=dtype), _empty(M, K, dtype=dtype), _empty(M)
    q, s = layer.forward(x, r, total=total, y=y, rstd=rstd)
    t, want_rstd, want = ref.norm(x, r, weight, 1e-5)
    # the sum in fp32, then in 16 bits: two roundings, of which the first is 2^-24 of the sum
    ref.check(total, x.double() + (0 if r is None else r.double()), t.double().abs() * 2.0 ** -24)
    _, want_rstd, want = ref.norm(total, None, weight, 1e-5)
    assert ((rstd.double() - want_rstd).abs() <= 2.0 ** -18 * want_rstd).all()
    ref.check(y, want, want.abs() * 2.0 ** -17, "y")
    ref.check_codes(q, s, want, want.abs() * 2.0 ** -17, "norm")
    # in place, and without the outputs that are not asked for
    again = x.clone() if r is None else r.clone()
    q2, s2 = layer.forward(again if r is None else x, r if r is None else again, total=again)
    assert torch.equal(again, total) and torch.equal(s2, s)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


def test_norm_of_strided_rows_and_without_codes():
    x = ref.activations(_gen(3), 6, 1024, torch.float16)
    weight = torch.ones(512, dtype=torch.float16, device="cuda")
    part = x[::2, 256:768]
    q, s = layers.RMSNorm(weight).forward(part)
    ref.check_codes(q, s, ref.norm(part, None, weight, 1e-6)[2],
                    ref.norm(part, None, weight, 1e-6)[2].abs() * 2.0 ** -17)
    y = _empty(3, 512, dtype=torch.float16)
    ql.qlinear_rmsnorm("float16", part, weight, 1e-6, 3, 512, y=y, ldx=2048)
    want = ref.norm(part, None, weight, 1e-6)[2]
    ref.check(y, want, want.abs() * 2.0 ** -17)


def test_norm_of_zeros():
    weight = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    q, s = layers.RMSNorm(weight).forward(torch.zeros(2, 256, dtype=torch.bfloat16, device="cuda"))
    assert (q.float() == 0).all() and (s == ref.FLOOR / ref.TOP).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,through,weight_too", [
    (1, 16, False, True), (1, 4096, True, True), (5, 144, True, True), (149, 2064, False, True),
    (601, 1024, True, True), (300, 8192, True, True), (299, 8208, False, True), (4, 16400, True, True),
    (3, 32768, True, True), (40, 512, True, False)])
def test_norm_backward(M, K, through, weight_too, dtype):
    gen = _gen(M + K)
    t = ref.activations(gen, M, K, dtype)
    weight = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(dtype)
    dy = (0.1 * torch.randn(M, K, generator=gen, device="cuda")).to(dtype)
    dt = (0.1 * torch.randn(M, K, generator=gen, device="cuda")).to(dtype) if through else None
    layer = layers.RMSNorm(weight, eps=1e-6)
    rstd = _empty(M)
    layer.forward(t, rstd=rstd)
    dweight = _empty(K) if weight_too else None
    dx = layer.backward(dy, t, rstd, dtotal=dt, dweight=dweight)
    want, err, want_w, err_w = ref.norm_backward(dy, t, rstd, weight, dt)
    ref.check(dx, want, err, "dx")
    if weight_too:
        off = (dweight.double() - want_w).abs()
        assert (off <= err_w).all(), (off / err_w).max().item()
    if through:  # in place, and the same bits again
        dx2 = layer.backward(dy, t, rstd, dtotal=dt, dx=dt)
        assert dx2 is dt and torch.equal(dx2, dx)
    dweight2 = _empty(K)
    layer.backward(dy, t, rstd, dweight=dweight2)
    if weight_too:
        assert torch.equal(dweight2, dweight)


def test_norm_gradient_against_differences():
    """dx and dweight against central differences of the norm in fp64, along random directions."""
    gen = _gen(8)
    M, K, eps = 3, 96, 1e-3
    x = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    weight = (1 + 0.2 * torch.randn(K, generator=gen, device="cuda")).to(torch.bfloat16)
    dy = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16)
    layer, rstd, dweight = layers.RMSNorm(weight, eps), _empty(M), _empty(K)
    layer.forward(x, rstd=rstd)
    dx = layer.backward(dy, x, rstd, dweight=dweight)

    def value(v, w):
        return (v * (v.square().mean(1, keepdim=True) + eps).rsqrt() * w * dy.double()).sum()

    h = 1e-5
    for seed in range(4):
        d = torch.randn(M, K, generator=_gen(seed), device="cuda").double()
        diff = (value(x.double() + h * d, weight.double()) -
                value(x.double() - h * d, weight.double())) / (2 * h)
        # dx is rounded to bf16: 2^-8 of each term; the difference's own error is about h^2
        assert abs((dx.double() * d).sum() - diff) <= (dx.double() * d).abs().sum() * 2.0 ** -8 + 1e-6
        d = torch.randn(K, generator=_gen(seed), device="cuda").double()
        diff = (value(x.double(), weight.double() + h * d) -
                value(x.double(), weight.double() - h * d)) / (2 * h)
        assert abs((dweight.double() * d).sum() - diff) <= \
            (dweight.double() * d).abs().sum() * 2.0 ** -18 + 1e-6


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("M,F", [(1, 16), (3, 144), (2, 2048), (33, 2064), (5, 14336)])
def test_gated(M, F, act, dtype):
    gu = ref.activations(_gen(M + F), M, 2 * F, dtype, 2.0)
    q, s = layers.fp8_gated(gu, act, q=_empty(M, F, dtype=F8), scales=_empty(M, ref.blocks(F)))
    h, err = ref.gated(gu, act)
    ref.check_codes(q, s, h, err, f"{M}x{F} {act}")
    dh = (0.1 * torch.randn(M, F, generator=_gen(F), device="cuda")).to(dtype)
    q, s = layers.fp8_gated_backward(dh, gu, act, q=_empty(M, 2 * F, dtype=F8),
                                     scales=_empty(M, ref.blocks(2 * F)))
    v, err = ref.gated_backward(dh, gu, act)
    ref.check_codes(q, s, v, err, f"{M}x{F} {act} backward")


# ---------------------------------------------------------------------------
# products

SHAPES = [(16, 16), (48, 144), (128, 128), (400, 272), (576, 1040), (1040, 528)]
ROWS = [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513]


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("N,K", SHAPES)
def test_linear(N, K, backward):
    gen = _gen(N + K)
    layer = layers.Fp8Linear(*ref.weights(gen, N, K))
    C, R = (N, K) if backward else (K, N)
    for M in ROWS:
        dtype = TYPES[M % 2]
        q, s = ref.quantize(torch.randn(M, C, generator=gen, device="cuda").double())
        out = _empty(M, R, dtype=dtype)
        (layer.backward if backward else layer.forward)(q, s, out)
        want, err = ref.product(q, s, layer.codes, layer.scales, backward)
        ref.check(out, want, err, f"{M} rows")
    assert layer.fused_read_error() == 0


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 12304, 2048), (40, 4096, 14336),
                                   (200, 8192, 4096), (1000, 4112, 4096), (2049, 2048, 8192),
                                   (4096, 1280, 1024)])
def test_linear_of_real_sizes(M, N, K, backward):
    gen = _gen(M + N + K)
    layer = layers.Fp8Linear(*ref.weights(gen, N, K))
    C = N if backward else K
    q, s = ref.quantize(ref.activations(gen, M, C, torch.float32).double())
    run = layer.backward if backward else layer.forward
    want, err = ref.product(q, s, layer.codes, layer.scales, backward)
    first = run(q, s, dtype=torch.float16)
    ref.check(first, want, err)
    for _ in range(3):  # what a call leaves in the workspace serves the next; the same bits
        assert torch.equal(run(q, s, dtype=torch.float16), first)
    assert layer.fused_read_error() == 0


@pytest.mark.parametrize("backward", [False, True], ids=["forward", "backward"])
@pytest.mark.parametrize("E,N,K,rows", [(1, 128, 128, 9), (4, 144, 272, 40), (7, 528, 400, 300),
                                        (16, 256, 512, 1500), (40, 400, 128, 90),
                                        (130, 48, 144, 700), (1024, 16, 32, 1200)])
def test_grouped(E, N, K, rows, backward):
    gen, rng = _gen(E + N), random.Random(E + K)
    layer = layers.Fp8Experts(*ref.weights(gen, E, N, K))
    C, R = (N, K) if backward else (K, N)
    run = layer.backward if backward else layer.forward
    splits = [ref.split(rows, E, rng), ref.split(rows, E, rng, empty=0.9),
              [0] * E + [rows], [0] + [rows] * E, [0] * (E + 1)]
    for k, at in enumerate(splits):
        lead, tail = (0, 0) if k == 0 else (3, 5)   # rows of nobody
        M = rows + lead + tail
        at = torch.tensor([a + lead for a in at], dtype=torch.int32, device="cuda")
        q, s = ref.quantize(torch.randn(M, C, generator=gen, device="cuda").double())
        out = _empty(M, R, dtype=TYPES[k % 2])
        before = out.clone()
        run(q, s, at, out)
        theirs = torch.zeros(M, dtype=torch.bool, device="cuda")
        for a, b, want, err in ref.grouped(q, s, at, layer.codes, layer.scales, backward):
            ref.check(out[a:b], want, err, f"split {k} rows {a}..{b}")
            theirs[a:b] = True
        assert torch.equal(out[~theirs].view(torch.int16), before[~theirs].view(torch.int16))
    assert layer.fused_read_error() == 0


def test_grouped_rows_of_others_are_not_read():
    """NaN in the rows of nobody, and in the rows of one expert, stays there."""
    gen = _gen(5)
    E, N, K, M = 3, 256, 384, 50
    layer = layers.Fp8Experts(*ref.weights(gen, E, N, K))
    q, s = ref.quantize(torch.randn(M, K, generator=gen, device="cuda").double())
    at = torch.tensor([4, 20, 31, 45], dtype=torch.int32, device="cuda")
    good = layer.forward(q, s, at, torch.zeros(M, N, dtype=torch.float16, device="cuda"))
    q = q.clone()
    q.view(torch.uint8)[:4] = 127
    q.view(torch.uint8)[20:31] = 127
    q.view(torch.uint8)[45:] = 127
    s = s.clone()
    s[:4] = s[45:] = float("nan")
    out = layer.forward(q, s, at, torch.zeros(M, N, dtype=torch.float16, device="cuda"))
    assert torch.isnan(out[20:31]).all()
    keep = [i for i in range(M) if not 20 <= i < 31]
    assert torch.equal(out[keep], good[keep])


def test_nan_codes_reach_their_outputs_only():
    gen = _gen(6)
    layer = layers.Fp8Linear(*ref.weights(gen, 256, 384))
    q, s = ref.quantize(torch.randn(70, 384, generator=gen, device="cuda").double())
    good = layer.forward(q, s)
    q.view(torch.uint8)[33, 130] = 255
    s[50, 2] = float("inf")
    out = layer.forward(q, s)
    assert torch.isnan(out[33]).all() and not torch.isfinite(out[50]).any()
    keep = [i for i in range(70) if i not in (33, 50)]
    assert torch.equal(out[keep], good[keep])


def test_bad_offsets_are_flagged_and_stay_inside():
    gen = _gen(7)
    E, N, K, M = 4, 128, 256, 24
    layer = layers.Fp8Experts(*ref.weights(gen, E, N, K))
    q, s = ref.quantize(torch.randn(M, K, generator=gen, device="cuda").double())
    for at, taken in (([0, 10, 5, 12, 24], [0, 10, 10, 12, 24]),
                      ([-7, 3, 9, 9, 100], [0, 3, 9, 9, 24]),
                      ([50, 60, 70, 2 ** 31 - 1, -2 ** 31], [24] * 5)):
        out = torch.zeros(M + 8, N, dtype=torch.bfloat16, device="cuda")
        layer.forward(q, s, torch.tensor(at, dtype=torch.int32, device="cuda"), out[:M])
        assert layer.fused_read_error() == 4
        assert (out[M:] == 0).all()
        for a, b, want, err in ref.grouped(q, s, torch.tensor(taken), layer.codes, layer.scales):
            ref.check(out[a:b], want, err)
    layer.forward(q, s, torch.tensor([0, 0, 8, 8, M], dtype=torch.int32, device="cuda"))
    assert layer.fused_read_error() == 0


# ---------------------------------------------------------------------------
# together


def _block(gen, E, H, F, dtype, norm=True):
    lead = (E,) if E else ()
    kind = layers.Fp8Experts if E else layers.Fp8Linear
    gate_up = kind(*layers.fp8_quantize_weights(
        (torch.randn(*lead, 2 * F, H, generator=gen, device="cuda") * 0.05).to(dtype)))
    down = kind(*layers.fp8_quantize_weights(
        (torch.randn(*lead, H, F, generator=gen, device="cuda") * 0.05).to(dtype)))
    weight = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
    return layers.Fp8GatedMLP(gate_up, down, layers.RMSNorm(weight) if norm else None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,M,H,F", [(0, 1, 256, 384), (0, 70, 512, 272), (0, 300, 1040, 640),
                                     (5, 37, 256, 144), (8, 500, 512, 384)])
def test_block_forward_and_backward(E, M, H, F, dtype):
    """Each step of the block against fp64, from the outputs of the step before it."""
    gen = _gen(M + F)
    block = _block(gen, E, H, F, dtype)
    x, r = (ref.activations(gen, M, H, dtype) for _ in range(2))
    rows = ()
    if E:
        rows = (torch.tensor(ref.split(M, E, random.Random(E)), dtype=torch.int32, device="cuda"),)
    total, rstd = _empty(M, H, dtype=dtype), _empty(M)
    gu = _empty(M, 2 * F, dtype=dtype)
    y = block.forward(x, r, *rows, total=total, rstd=rstd, gu=gu)

    def product(layer, q, s, backward, out):
        if not E:
            want, err = ref.product(q, s, layer.codes, layer.scales, backward)
            return ref.check(out, want, err)
        for a, b, want, err in ref.grouped(q, s, rows[0], layer.codes, layer.scales, backward):
            ref.check(out[a:b], want, err)

    q, s = block.norm.forward(x, r)
    product(block.gate_up, q, s, False, gu)
    product(block.down, *layers.fp8_gated(gu, "silu"), False, y)

    dy, dt = ((0.1 * torch.randn(M, H, generator=gen, device="cuda")).to(dtype) for _ in range(2))
    dweight = _empty(H)
    dx = block.backward(dy, gu, total, rstd, *rows, dtotal=dt, dweight=dweight)
    q, s = layers.fp8_quantize(dy)
    dh = block.down.backward(q, s, *rows, dtype=dtype)
    product(block.down, q, s, True, dh)
    q, s = layers.fp8_gated_backward(dh, gu, "silu")
    dv = block.gate_up.backward(q, s, *rows, dtype=dtype)
    product(block.gate_up, q, s, True, dv)
    want, err, want_w, err_w = ref.norm_backward(dv, total, rstd, block.norm.weight, dt)
    ref.check(dx, want, err)
    assert ((dweight.double() - want_w).abs() <= err_w).all()
    assert block.gate_up.fused_read_error() == 0 and block.down.fused_read_error() == 0


def test_block_without_a_norm_and_its_refusals():
    gen = _gen(2)
    block = _block(gen, 0, 256, 128, torch.bfloat16, norm=False)
    x = ref.activations(gen, 20, 256, torch.bfloat16)
    gu = _empty(20, 256, dtype=torch.bfloat16)
    y = block.forward(x, gu=gu)
    q, s = layers.fp8_quantize(x)
    want, err = ref.product(q, s, block.gate_up.codes, block.gate_up.scales)
    ref.check(gu, want, err)
    dx = block.backward(y, gu)
    assert dx.shape == x.shape and torch.isfinite(dx).all()
    for kw in (dict(residual=x), dict(rstd=_empty(20)),
               dict(offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            block.forward(x, **kw)


def test_calls_without_rows():
    gen = _gen(2)
    block = _block(gen, 3, 256, 128, torch.bfloat16)
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    gu, rstd, dweight = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), _empty(0), _empty(256)
    assert block.forward(x, offsets=at, rstd=rstd, gu=gu).shape == (0, 256)
    assert block.backward(x, gu, x, rstd, at, dweight=dweight).shape == (0, 256)
    assert (dweight == 0).all()


def test_arguments_are_checked():
    gen = _gen(1)
    layer = layers.Fp8Linear(*ref.weights(gen, 64, 128))
    q, s = ref.quantize(torch.randn(4, 128, generator=gen, device="cuda").double())
    for bad in (dict(q=q[:, :64]), dict(q=q.float()), dict(scales=s[:3]), dict(scales=s.half()),
                dict(y=_empty(4, 64)), dict(y=_empty(4, 32, dtype=torch.float16)),
                dict(q=q.cpu()), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            layer.forward(**{"q": q, "scales": s, **bad})
    experts = layers.Fp8Experts(*ref.weights(gen, 2, 64, 128))
    for at in (torch.zeros(3, dtype=torch.int64, device="cuda"),
               torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32)):
        with pytest.raises(ValueError):
            experts.forward(q, s, at)
    x = torch.randn(4, 256, generator=gen, device="cuda").half()
    for f in (lambda: layers.fp8_quantize(x.float()), lambda: layers.fp8_quantize(x.t()),
              lambda: layers.fp8_quantize(x[0]), lambda: layers.fp8_gated(x[:, 1:]),
              lambda: layers.fp8_gated(x[:, :255]),
              lambda: layers.fp8_quantize(x.clone().requires_grad_()),
              lambda: layers.fp8_gated_backward(x, x),
              lambda: layers.RMSNorm(x[0]).forward(x.bfloat16()),
              lambda: layers.RMSNorm(x[0]).forward(x, residual=x[:2])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(ql.QLinearError):
        layers.fp8_quantize(x[:, :24].contiguous())
