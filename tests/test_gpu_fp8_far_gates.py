"""Gates at the far ends of bf16's range: the activations and their derivatives are what they tend
to, on the GPU."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import fp8_ref as ref
    from weight_only_quantized_gemv_b200 import layers

SIZES = [3.0, 40.0, 1e4, 1e13, 2e19, 1e20, 1e30, 3e38]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("F", [128 * len(SIZES), 136 * len(SIZES)])
def test_far_gates(F, act):
    """A size of gate to each run of columns, both signs; the factors are at most one."""
    M, gen = 4, torch.Generator(device="cuda").manual_seed(F)
    run = F // len(SIZES)
    size = torch.tensor(SIZES, device="cuda").repeat_interleave(run)
    sign = torch.where(torch.rand(M, F, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
    g = (sign * size).bfloat16()
    u, dh = ((2 * torch.rand(M, F, generator=gen, device="cuda") - 1).bfloat16() for _ in range(2))
    gu = torch.cat([g, u], 1)
    assert bool(torch.isfinite(gu).all())
    want, err = ref.gated(gu, act)
    ref.check_codes(*layers.fp8_gated(gu, act), want, err, f"{act} forward")
    want, err = ref.gated_backward(dh, gu, act)
    assert bool(torch.isfinite(want).all())
    q, s = layers.fp8_gated_backward(dh, gu, act)
    assert bool(torch.isfinite(s).all()) and bool(torch.isfinite(q.float()).all())
    ref.check_codes(q, s, want, err, f"{act} backward")
