"""The measured operators: quantized linear layers with a fused epilogue, the gated
feed-forward projection, and their backward passes through the frozen quantized weights.

Four operators, on the dense weight formats (W2 / W4 / W8 with a scale and a zero per 128
weights of a column, LUT4 with a 16-entry table and an absmax per 64), fp16 activations:

  linear           z = x W + bias;  y = act(z) + residual          (z is kept for training)
  linear_backward  dz = dy act'(z);  dx = dz W^T;  dbias = sum of dz over the rows
  gated            g = x Wg + bg, u = x Wu + bu;  h = act(g) u     (g, u kept for training)
  gated_backward   dg = dh u act'(g), du = dh act(g);  dx = dg Wg^T + du Wu^T;
                   dbias = sums of dg and du over the rows

``run`` computes them with elementary torch operations in fp32 (``own`` false) or through
the framework's layers (``own`` true); ``exact`` in fp64.
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
GROUP, BLOCK = 128, 64
BITS = {"w2": 2, "w4": 4, "w8": 8, "lut4": 4}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # attention output projection while decoding one sequence, added to the residual
        {"name": "linear-w4-m1", "op": "linear", "fmt": "w4", "M": 1, "K": 4096, "N": 4096,
         "act": "none", "bias": False, "residual": True, "save": False},
        # query / key / value projection with a bias while decoding a batch of 24
        {"name": "linear-w8-m24", "op": "linear", "fmt": "w8", "M": 24, "K": 4096, "N": 12288,
         "act": "none", "bias": True, "residual": False, "save": False},
        # down projection of a short prompt, added to the residual
        {"name": "linear-lut4-m200", "op": "linear", "fmt": "lut4", "M": 200, "K": 14336,
         "N": 4096, "act": "none", "bias": False, "residual": True, "save": False},
        # up projection with bias and GELU over a training batch, pre-activation kept
        {"name": "linear-w4-m2048", "op": "linear", "fmt": "w4", "M": 2048, "K": 8192,
         "N": 28672, "act": "gelu", "bias": True, "residual": False, "save": True},
        # gate and up projections while decoding one sequence
        {"name": "gated-w4-m1", "op": "gated", "fmt": "w4", "M": 1, "K": 4096, "F": 14336,
         "act": "silu", "bias": False, "save": False},
        # ... a batch of 13 with 2-bit weights
        {"name": "gated-w2-m13", "op": "gated", "fmt": "w2", "M": 13, "K": 8192, "F": 14336,
         "act": "silu", "bias": True, "save": False},
        # ... a training batch of odd length, gate and up kept
        {"name": "gated-w4-m513", "op": "gated", "fmt": "w4", "M": 513, "K": 4096, "F": 14336,
         "act": "silu", "bias": False, "save": True},
        # backward of a square projection, a short sequence
        {"name": "linear_backward-w4-m96", "op": "linear_backward", "fmt": "w4", "M": 96,
         "K": 4096, "N": 4096, "act": "none", "dbias": True},
        # ... of a projection with ReLU, 8-bit weights, odd length
        {"name": "linear_backward-w8-m777", "op": "linear_backward", "fmt": "w8", "M": 777,
         "K": 4096, "N": 12288, "act": "relu", "dbias": True},
        # ... of the largest layer over a training batch
        {"name": "linear_backward-w4-m2048", "op": "linear_backward", "fmt": "w4", "M": 2048,
         "K": 8192, "N": 28672, "act": "gelu", "dbias": True},
        # backward of the gated projection, a short sequence on a narrow layer of ragged width
        {"name": "gated_backward-lut4-m65", "op": "gated_backward", "fmt": "lut4", "M": 65,
         "K": 2048, "F": 1168, "act": "gelu_tanh", "dbias": False},
        # ... over a training batch
        {"name": "gated_backward-w4-m1024", "op": "gated_backward", "fmt": "w4", "M": 1024,
         "K": 4096, "F": 14336, "act": "silu", "dbias": False},
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear", "gated", "linear_backward", "gated_backward"])
    case = {"op": op, "fmt": rng.choice(["w2", "w4", "w8", "lut4"]),
            "M": log_uniform(1, 2048), "K": 128 * log_uniform(1, 64)}
    if op.startswith("linear"):
        case["N"] = 16 * log_uniform(1, 1792)
        case["act"] = rng.choice(ACTS)
    else:
        case["F"] = 16 * log_uniform(1, 896)
        case["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    if op.endswith("backward"):
        case["dbias"] = rng.random() < 0.5
    else:
        case["bias"] = rng.random() < 0.5
        case["save"] = rng.random() < 0.5
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return case


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEVICE) * std


def _quantized(gen, fmt, K, N):
    """Weights N(0, 0.02) in the format: codes uint8 [K, N] and the two parameter arrays
    (fp16 scales and zeros [K / 128, N], or the fp16 table [16] and fp32 absmax [K / 64, N])."""
    w = _normal(gen, K, N, std=0.02)
    if fmt == "lut4":
        inner = torch.rand(13, generator=gen, device=DEVICE) * 2 - 1
        table = torch.cat([inner, torch.tensor([-1.0, 0.0, 1.0], device=DEVICE)])
        table = table.sort().values.half()
        absmax = w.view(K // BLOCK, BLOCK, N).abs().amax(1)
        unit = w.view(K // BLOCK, BLOCK, N).div_(absmax.unsqueeze(1)).view(K, N)
        edges = (table[1:].float() + table[:-1].float()) / 2
        return torch.bucketize(unit, edges).to(torch.uint8), table, absmax
    top = float((1 << BITS[fmt]) - 1)
    wg = w.view(K // GROUP, GROUP, N)
    low, high = wg.amin(1), wg.amax(1)
    scale = ((high - low) / top).half()
    s = scale.float()
    zero = (-low / s).round().clamp(0, top)
    codes = wg.div_(s.unsqueeze(1)).round_().add_(zero.unsqueeze(1)).clamp_(0, top)
    return codes.to(torch.uint8).view(K, N), scale, zero.half()


def _canonical(fmt, codes):
    """The framework's canonical code layout: int32 words of 32 / bits codes along K, or for
    LUT4 bytes of two codes (low half = even k)."""
    K, N = codes.shape
    if fmt == "lut4":
        pair = codes.view(K // 2, 2, N)
        return pair[:, 0] | (pair[:, 1] << 4)
    per = 32 // BITS[fmt]
    fields = codes.view(K // per, per, N)
    words = torch.zeros(K // per, N, dtype=torch.int32, device=codes.device)
    for i in range(per):
        words |= fields[:, i].to(torch.int32) << (BITS[fmt] * i)
    return words


def _inputs(case, seed):
    """(weights, tensors): one quantized matrix, or the gate's and the up projection's, as
    (codes, p0, p1), and the activations of the case."""
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, fmt, M, K = case["op"], case["fmt"], case["M"], case["K"]
    gated = op.startswith("gated")
    width = case["F"] if gated else case["N"]
    weights = [_quantized(gen, fmt, K, width) for _ in range(2 if gated else 1)]
    if gated and fmt == "lut4":  # one table for both
        weights[1] = (weights[1][0], weights[0][1], weights[1][2])
    lead = (2, width) if gated else (width,)
    t = {}
    if op.endswith("backward"):
        t["dy"] = _normal(gen, M, width, std=0.25).half()
        t["z"] = _normal(gen, M, *lead, std=0.02 * math.sqrt(K)).half()
    else:
        t["x"] = _normal(gen, M, K).half()
        if case["bias"]:
            t["bias"] = _normal(gen, *lead, std=0.1).half()
        if case.get("residual"):
            t["residual"] = _normal(gen, M, width).half()
    return weights, t


def prepare(case, seed):
    weights, t = _inputs(case, seed)
    state = dict(case, **{"t": t})
    fmt, M, K = case["fmt"], case["M"], case["K"]
    stored = [(_canonical(fmt, c), p0, p1) for c, p0, p1 in weights]
    if not own:
        state["weights"] = stored
        return state
    import weight_only_quantized_gemv_b200 as ql
    from weight_only_quantized_gemv_b200 import layers

    host = [(c.cpu().numpy().view(np.uint8 if fmt == "lut4" else np.uint32),
             p0.cpu().numpy(), p1.cpu().numpy()) for c, p0, p1 in stored]
    if case["op"].startswith("gated"):
        state["layer"] = layers.GatedLinear(ql.FORMATS[fmt], K, case["F"], host[0], host[1],
                                            device=DEVICE)
    else:
        state["layer"] = layers.QuantLinear(ql.FORMATS[fmt], K, case["N"], *host[0],
                                            device=DEVICE)
    state["layer"].reserve(M)
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    layer, t, op, M, K = s["layer"], s["t"], s["op"], s["M"], s["K"]
    if op == "linear":
        z = None
        if s["save"]:
            z = torch.empty((M, s["N"]), dtype=torch.float16, device=DEVICE)
        y = layer.linear(t["x"], bias=t.get("bias"), residual=t.get("residual"), act=s["act"],
                         z=z)
        return (y,) if z is None else (y, z)
    if op == "gated":
        gu = None
        if s["save"]:
            gu = torch.empty((M, 2, s["F"]), dtype=torch.float16, device=DEVICE)
        h = layer.forward(t["x"], bias=t.get("bias"), act=s["act"], gu=gu)
        return (h,) if gu is None else (h, gu)
    dbias = None
    if op == "linear_backward":
        if s["dbias"]:
            dbias = torch.empty((s["N"],), dtype=torch.float32, device=DEVICE)
        dx = layer.linear_backward(t["dy"], z=None if s["act"] == "none" else t["z"],
                                   act=s["act"], dbias=dbias)
    else:
        if s["dbias"]:
            dbias = torch.empty((2, s["F"]), dtype=torch.float32, device=DEVICE)
        dx = layer.backward(t["dy"], t["z"], act=s["act"], dbias=dbias)
    return (dx,) if dbias is None else (dx, dbias)


def _dequantize(fmt, words, p0, p1):
    """fp32 weights [K, N] from the stored codes."""
    if fmt == "lut4":
        codes = torch.stack([words & 15, words >> 4], 1).view(-1, words.shape[1])
        K, N = codes.shape
        w = p0.float()[codes.int()].view(K // BLOCK, BLOCK, N)
        return (w * p1.unsqueeze(1)).view(K, N)
    bits = BITS[fmt]
    codes = torch.stack([(words >> (bits * i)) & ((1 << bits) - 1)
                         for i in range(32 // bits)], 1)
    K, N = codes.shape[0] * codes.shape[1], words.shape[1]
    q = codes.view(K // GROUP, GROUP, N).float()
    return ((q - p1.float().unsqueeze(1)) * p0.float().unsqueeze(1)).view(K, N)


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return z * (z > 0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * density
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * c * (1 + 3 * 0.044715 * z * z)
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _run_plain(s):
    t, op, act = s["t"], s["op"], s["act"]
    w = [_dequantize(s["fmt"], *stored) for stored in s["weights"]]
    if op == "linear":
        z = t["x"].float() @ w[0]
        if s["bias"]:
            z = z + t["bias"].float()
        y = _act(act, z)
        if s["residual"]:
            y = y + t["residual"].float()
        return (y.half(), z.half()) if s["save"] else (y.half(),)
    if op == "gated":
        x = t["x"].float()
        gu = torch.stack([x @ w[0], x @ w[1]], 1)
        if s["bias"]:
            gu = gu + t["bias"].float()
        h = (_act(act, gu[:, 0]) * gu[:, 1]).half()
        return (h, gu.half()) if s["save"] else (h,)
    dy = t["dy"].float()
    if op == "linear_backward":
        dz = dy * _act_grad(act, t["z"].float()) if act != "none" else dy
        dx = (dz @ w[0].t()).half()
    else:
        g, u = t["z"][:, 0].float(), t["z"][:, 1].float()
        dz = torch.stack([dy * u * _act_grad(act, g), dy * _act(act, g)], 1)
        dx = (dz[:, 0] @ w[0].t() + dz[:, 1] @ w[1].t()).half()
    return (dx, dz.sum(0)) if s["dbias"] else (dx,)


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_act(name, z, order):
    """The activation (order 0) or its derivative (order 1)."""
    if name == "none":
        return z.clone() if order == 0 else torch.full_like(z, 1.0)
    if name == "relu":
        return z.clamp_min(0.0) if order == 0 else (z > 0).double()
    if name == "silu":
        sig = torch.sigmoid(z)
        return z * sig if order == 0 else sig + z * sig * torch.sigmoid(-z)
    if name == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf if order == 0 else cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    # gelu_tanh: (1 + tanh(v)) / 2 = sigmoid(2 v)
    a = math.sqrt(2.0 / math.pi)
    sig = torch.sigmoid(2.0 * a * (z + 0.044715 * z ** 3))
    if order == 0:
        return z * sig
    return sig + z * sig * (1.0 - sig) * 2.0 * a * (1.0 + 0.134145 * z ** 2)


def _exact_weight(fmt, codes, p0, p1):
    if fmt == "lut4":
        return p0.double()[codes.long()] * p1.double().repeat_interleave(BLOCK, 0)
    zero = p1.double().repeat_interleave(GROUP, 0)
    return (codes.double() - zero) * p0.double().repeat_interleave(GROUP, 0)


def exact(case, seed):
    weights, t = _inputs(case, seed)
    op, fmt, act = case["op"], case["fmt"], case["act"]
    t = {k: v.double() for k, v in t.items()}

    def columns(codes, p0, p1):
        """(slice, fp64 weights) of up to 4096 columns at a time."""
        for c0 in range(0, codes.shape[1], 4096):
            sl = slice(c0, c0 + 4096)
            yield sl, _exact_weight(fmt, codes[:, sl], p0 if fmt == "lut4" else p0[:, sl],
                                    p1[:, sl])

    def product(x, weight):
        return torch.cat([x @ w for _, w in columns(*weight)], 1)

    def product_t(d, weight):
        total = torch.zeros(d.shape[0], case["K"], dtype=torch.float64, device=d.device)
        for sl, w in columns(*weight):
            total += torch.einsum("mn,kn->mk", d[:, sl], w)
        return total

    if op == "linear":
        z = product(t["x"], weights[0])
        if "bias" in t:
            z += t["bias"]
        y = _exact_act(act, z, 0)
        if "residual" in t:
            y += t["residual"]
        return (y, z) if case["save"] else (y,)
    if op == "gated":
        g, u = (product(t["x"], w) for w in weights)
        if "bias" in t:
            g, u = g + t["bias"][0], u + t["bias"][1]
        h = _exact_act(act, g, 0) * u
        return (h, torch.stack([g, u], 1)) if case["save"] else (h,)
    if op == "linear_backward":
        dz = t["dy"] * _exact_act(act, t["z"], 1)
        dx, db = product_t(dz, weights[0]), dz.sum(0)
    else:
        g, u = t["z"].unbind(1)
        dg, du = t["dy"] * u * _exact_act(act, g, 1), t["dy"] * _exact_act(act, g, 0)
        dx = product_t(dg, weights[0]) + product_t(du, weights[1])
        db = torch.stack([dg.sum(0), du.sum(0)])
    return (dx, db) if case["dbias"] else (dx,)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op, fmt, M, K = case["op"], case["fmt"], case["M"], case["K"]
    gated = op.startswith("gated")
    N = 2 * case["F"] if gated else case["N"]      # columns of the weights
    width = case["F"] if gated else case["N"]      # of the layer's output
    if fmt == "lut4":
        weight = K * N // 2 + 4 * (K // BLOCK) * N + 32
    else:
        weight = K * N * BITS[fmt] // 8 + 4 * (K // GROUP) * N
    if op.endswith("backward"):
        read = 2 * M * width + (2 * M * N if gated or case["act"] != "none" else 0)
        written = 2 * M * K + (4 * N if case["dbias"] else 0)
    else:
        read = 2 * M * K + (2 * N if case["bias"] else 0)
        read += 2 * M * N if case.get("residual") else 0
        written = 2 * M * width + (2 * M * N if case["save"] else 0)
    return {"bytes": weight + read + written, "flops": 2 * M * N * K}
