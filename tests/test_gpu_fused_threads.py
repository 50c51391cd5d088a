"""The fused layers called from several host threads, on the GPU."""
import copy
import threading
import time

import pytest

from synth import gen
from tests import fused_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    torch.cuda.set_device(0)


def _t(seed, *shape, std=1.0):
    return torch.from_numpy(ref.seeded(seed, *shape, std=std)).to(DEV)


def _run(threads):
    errors = []

    def guard(fn):
        try:
            torch.cuda.set_device(0)
            fn()
        except BaseException as e:  # noqa: BLE001 - reported below
            errors.append(e)

    ts = [threading.Thread(target=guard, args=(f,)) for f in threads]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("streams", [1, 2])
def test_enqueueing_is_exclusive(streams):
    """Two threads call one layer: neither enters the library while the other is in it, and the
    stream that comes second waits for all that the first was given."""
    lay = layers.from_uniform(gen.uniform_layer(1, 384, 208, 4), DEV)
    lay.reserve(4)
    x = _t(1, 4, 384)
    lay.linear(x)
    st = [torch.cuda.Stream() for _ in range(streams)]
    inside, most, order = [0], [0], []

    def entry(*args):
        inside[0] += 1
        most[0] = max(most[0], inside[0])
        order.append(args[-1])
        time.sleep(0.002)  # the interpreter lock is free, as during the library's call
        inside[0] -= 1
        return 0

    switches = []
    orig = lay._fused_switch
    lay._fused_switch = lambda raw, s: (switches.append((raw, inside[0])), orig(raw, s))

    def caller(s):
        for _ in range(20):
            lay._fused_call(entry, "entry", (), 4, False, None, s)

    _run([lambda: caller(st[0]), lambda: caller(st[-1])])
    assert len(order) == 40 and most[0] == 1
    assert all(n == 0 for _, n in switches)  # no switch while the other's call is under way
    # every change of stream was a switch, in the calls' order
    raws = [r for i, r in enumerate(order) if i == 0 or order[i - 1] != r]
    assert [r for r, _ in switches] == raws


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("streams", [1, 4])
def test_threads_get_their_own_results(M, streams):
    """Four threads, forward and backward calls with inputs of their own, on one stream (a
    backward call is several launches) or on one each."""
    K, F = 2048, 592
    raw = [gen.uniform_layer(s, K, F, 4) for s in (2, 3)]
    lay = layers.GatedLinear(ql.QL_FMT_W4, K, F, *[(u.qweight, u.scales, u.zeros) for u in raw],
                             device=DEV)
    lay.reserve(M)
    args = [(_t(10 + i, M, K), _t(20 + i, M, F, std=0.25), _t(30 + i, M, 2, F)) for i in range(4)]

    def calls(i, stream=None):
        x, dh, gu = args[i]
        db = torch.empty((2, F), dtype=torch.float32, device=DEV)
        return (lay.forward(x, stream=stream),
                lay.backward(dh, gu, dbias=db, stream=stream), db)

    want = [calls(i) for i in range(4)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(streams)]
    got = [[] for _ in range(4)]

    def caller(i):
        s = st[i % streams]
        with torch.cuda.stream(s):
            for _ in range(25):
                got[i].append(calls(i, s))

    _run([lambda i=i: caller(i) for i in range(4)])
    torch.cuda.synchronize()
    for i in range(4):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i])), i
    assert lay.fused_read_error() == 0


def test_a_copied_layer_has_a_lock_of_its_own():
    lay = layers.from_uniform(gen.uniform_layer(1, 384, 208, 4), DEV)
    x = _t(1, 4, 384)
    want = lay.linear(x)
    for other in (copy.deepcopy(lay), copy.copy(lay)):
        assert other._fused_lock is not lay._fused_lock and not other._fused_ws
        assert torch.equal(other.linear(x), want)
