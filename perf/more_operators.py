"""The measured operators of the 8-bit floating-point path: what lies between the residual stream
and the residual stream of a feed-forward block whose products have both operands in e4m3.

  norm             t = x + residual, rounded to the stream's type;  r = 1 / sqrt(mean(t^2) + eps);
                   y = t r w;  codes and scales of y
  norm_backward    dx = r (w dy - t r^2 mean(w dy t)) + dt;  dw = sum of dy t r over the rows
  gated            h = act(g) u;  codes and scales of h
  gated_backward   dg = dh u act'(g), du = dh act(g);  codes and scales of (dg, du)
  linear           y = X W^T of coded X [M, K] and W [N, K]
  linear_backward  dx = D W of coded D [M, N]
  grouped          rows offsets[e] .. offsets[e + 1] of X times the matrix of expert e
  grouped_backward the same rows of D times the matrix of expert e

Codes of a tensor's rows: for each 128 columns (the last block may be shorter) scale = max|v| / 448
and e4m3(v / scale), 448 being the type's largest value.  Weights have one scale per 128 x 128
block.  Codes are returned as the 8-bit floating-point numbers that they are, beside their scales.

``run`` computes the operators with elementary torch operations in fp32 (``own`` false) or through
the framework's layers (``own`` true); ``exact`` in fp64.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 128
TOP = 448.0            # the largest e4m3 value
FLOOR = 2.0 ** -100    # a block's largest value is taken as at least this
EPS = 1e-6
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def listed():
    return [
        # the norm before a layer while decoding one sequence
        {"name": "norm-m1", "op": "norm", "type": "bf16", "M": 1, "K": 4096, "residual": True,
         "save": False, "dense": False},
        # ... over a prompt or a training batch, statistics and the 16-bit values kept
        {"name": "norm-m4096", "op": "norm", "type": "bf16", "M": 4096, "K": 8192,
         "residual": True, "save": True, "dense": True},
        # its backward pass over a batch of odd length
        {"name": "norm_backward-m2047", "op": "norm_backward", "type": "bf16", "M": 2047,
         "K": 8192, "through": True},
        # gate and up values of a decoding batch on their way into the down product
        {"name": "gated-m24", "op": "gated", "type": "f16", "M": 24, "F": 14336, "act": "silu"},
        # gradients of a training batch's gate and up values on their way into the backward product
        {"name": "gated_backward-m1024", "op": "gated_backward", "type": "bf16", "M": 1024,
         "F": 14336, "act": "silu"},
        # attention output projection while decoding one sequence
        {"name": "linear-m1", "op": "linear", "type": "bf16", "M": 1, "K": 4096, "N": 4096},
        # up projection for a decoding batch
        {"name": "linear-m33", "op": "linear", "type": "f16", "M": 33, "K": 8192, "N": 28672},
        # ... for a training batch or a long prompt
        {"name": "linear-m4096", "op": "linear", "type": "bf16", "M": 4096, "K": 8192, "N": 28672},
        # backward of a projection of ragged width, odd length
        {"name": "linear_backward-m777", "op": "linear_backward", "type": "bf16", "M": 777,
         "K": 4096, "N": 12304},
        # experts' up projections for a decoding batch: a few rows each, some experts without
        {"name": "grouped-e64-t40", "op": "grouped", "type": "bf16", "E": 64, "active": 23,
         "T": 40, "K": 4096, "N": 2048},
        # ... for a long prompt: hundreds of rows each, ragged
        {"name": "grouped-e64-t16384", "op": "grouped", "type": "bf16", "E": 64, "active": 62,
         "T": 16384, "K": 4096, "N": 2048},
        # backward of a few large experts over a batch of odd length
        {"name": "grouped_backward-e8-t2049", "op": "grouped_backward", "type": "f16", "E": 8,
         "active": 8, "T": 2049, "K": 4096, "N": 14336},
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "norm_backward", "gated", "gated_backward", "linear",
                     "linear_backward", "grouped", "grouped_backward"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"])}
    if op.startswith("norm"):
        case.update(M=log_uniform(1, 4096), K=16 * log_uniform(8, 512))
        if op == "norm":
            case.update(residual=rng.random() < 0.7, save=rng.random() < 0.5,
                        dense=rng.random() < 0.5)
        else:
            case["through"] = rng.random() < 0.5
    elif op.startswith("gated"):
        case.update(M=log_uniform(1, 2048), F=16 * log_uniform(8, 896), act=rng.choice(ACTS))
    elif op.startswith("linear"):
        case.update(M=log_uniform(1, 4096), K=16 * log_uniform(8, 512),
                    N=16 * log_uniform(8, 1792))
    else:
        E = log_uniform(2, 64)
        T = log_uniform(1, 16384)
        # up to the listed cases' weights, and their flops
        K = 16 * log_uniform(8, 256)
        N = 16 * log_uniform(8, min(896, max(9, 2048 * 256 * 64 // (16 * 16 * E * (K // 16)))))
        case.update(E=E, active=rng.randint(1, min(E, T)), T=T, K=K, N=N)
        if op == "grouped" and rng.random() < 0.5:
            case["T"] = min(T, 4 * E)
            case["active"] = min(case["active"], case["T"])
    return case


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEVICE) * std


def _blocks(v):
    """[..., C] -> [..., blocks, 128], the last block filled up with zeros."""
    C = v.shape[-1]
    return torch.nn.functional.pad(v, (0, -C % BLOCK)).unflatten(-1, (-1, BLOCK))


def _coded_rows(v):
    """(codes, scales [..., blocks]) of fp32 rows."""
    blocks = _blocks(v)
    scale = blocks.abs().amax(-1).clamp_min(FLOOR) / TOP
    q = (blocks / scale.unsqueeze(-1)).clamp(-TOP, TOP).flatten(-2)[..., :v.shape[-1]]
    return q.to(torch.float8_e4m3fn), scale


def _spread(scales, rows, cols):
    """Scales [..., rows / 128, cols / 128] for each weight."""
    full = scales.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)
    return full[..., :rows, :cols]


def _weights(gen, *shape):
    """(codes [..., N, K], scales [..., N / 128, K / 128]) of weights N(0, 0.02)."""
    N, K = shape[-2:]
    w = _normal(gen, *shape, std=0.02)
    tiles = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    tiles = tiles.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))
    scale = tiles.abs().amax((-3, -1)) / TOP
    del tiles
    w /= _spread(scale, N, K)
    return w.clamp_(-TOP, TOP).to(torch.float8_e4m3fn), scale


def _activations(gen, M, K, std=1.0):
    """Values whose columns differ in size, as the channels of a hidden state do."""
    return _normal(gen, M, K) * torch.exp(_normal(gen, K, std=0.5)) * std


def _offsets(gen, case):
    """Row ranges of the experts, int32 [E + 1]: `active` of them have rows, one to several times
    the average."""
    E, A, T = case["E"], case["active"], case["T"]
    share = torch.rand(A, generator=gen, device=DEVICE).mul_(1.5).add_(0.5)
    ends = (share.cumsum(0) / share.sum() * (T - A)).round().long()
    counts = torch.diff(ends, prepend=ends.new_zeros(1)) + 1
    counts[-1] += T - counts.sum()
    per = torch.zeros(E, dtype=torch.long, device=DEVICE)
    per[torch.randperm(E, generator=gen, device=DEVICE)[:A]] = counts
    return torch.nn.functional.pad(per.cumsum(0), (1, 0)).to(torch.int32)


def _inputs(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    op, dtype = case["op"], TYPES[case["type"]]
    t = {}
    if op.startswith("norm"):
        M, K = case["M"], case["K"]
        t["weight"] = (1 + _normal(gen, K, std=0.2)).to(dtype)
        t["x"] = _activations(gen, M, K).to(dtype)
        if op == "norm_backward":
            t["rstd"] = (t["x"].double().square().mean(1) + EPS).rsqrt().float()
            t["dy"] = _normal(gen, M, K, std=0.05).to(dtype)
            if case["through"]:
                t["dt"] = _normal(gen, M, K, std=0.05).to(dtype)
        elif case["residual"]:
            t["residual"] = _activations(gen, M, K, std=3.0).to(dtype)
    elif op.startswith("gated"):
        M, F = case["M"], case["F"]
        t["gu"] = _activations(gen, M, 2 * F).to(dtype)
        if op == "gated_backward":
            t["dh"] = _normal(gen, M, F, std=0.05).to(dtype)
    else:
        rows, K, N = case.get("M", case.get("T")), case["K"], case["N"]
        if op.startswith("grouped"):
            t["offsets"] = _offsets(gen, case)
            t["codes"], t["wscale"] = _weights(gen, case["E"], N, K)
        else:
            t["codes"], t["wscale"] = _weights(gen, N, K)
        if op.endswith("backward"):
            t["q"], t["scale"] = _coded_rows(_normal(gen, rows, N, std=0.05))
        else:
            t["q"], t["scale"] = _coded_rows(_activations(gen, rows, K))
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    state = dict(case, t=t, dtype=TYPES[case["type"]])
    op = case["op"]
    if op.startswith("grouped"):
        state["most"] = int(torch.diff(t["offsets"]).max())
    if own:
        from weight_only_quantized_gemv_b200 import layers

        if op.startswith("norm"):
            state["layer"] = layers.RMSNorm(t["weight"], eps=EPS)
            if op == "norm_backward":
                state["layer"].reserve(case["M"])
        elif op.startswith("linear"):
            state["layer"] = layers.Fp8Linear(t["codes"], t["wscale"])
            state["layer"].reserve(case["M"])
        elif op.startswith("grouped"):
            state["layer"] = layers.Fp8Experts(t["codes"], t["wscale"])
            state["layer"].reserve(case["T"])
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from weight_only_quantized_gemv_b200 import layers

    t, op, layer, dtype = s["t"], s["op"], s.get("layer"), s["dtype"]
    if op == "norm":
        x = t["x"]
        total = torch.empty_like(x) if s["residual"] else None
        y = torch.empty_like(x) if s["dense"] else None
        rstd = x.new_empty(x.shape[0], dtype=torch.float32) if s["save"] else None
        q, scale = layer.forward(x, residual=t.get("residual"), total=total, y=y, rstd=rstd)
        return {"q": q, "scale": scale, "total": total, "y": y, "rstd": rstd}
    if op == "norm_backward":
        dweight = torch.empty(s["K"], dtype=torch.float32, device=DEVICE)
        dx = layer.backward(t["dy"], t["x"], t["rstd"], dtotal=t.get("dt"), dweight=dweight)
        return {"dx": dx, "dweight": dweight}
    if op == "gated":
        q, scale = layers.fp8_gated(t["gu"], act=s["act"])
        return {"q": q, "scale": scale}
    if op == "gated_backward":
        q, scale = layers.fp8_gated_backward(t["dh"], t["gu"], act=s["act"])
        return {"q": q, "scale": scale}
    if op == "linear":
        return {"y": layer.forward(t["q"], t["scale"], dtype=dtype)}
    if op == "linear_backward":
        return {"dx": layer.backward(t["q"], t["scale"], dtype=dtype)}
    if op == "grouped":
        return {"y": layer.forward(t["q"], t["scale"], t["offsets"], dtype=dtype)}
    return {"dx": layer.backward(t["q"], t["scale"], t["offsets"], dtype=dtype)}


def _act(name, z):
    if name == "relu":
        return z * (z > 0)
    if name == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if name == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        density = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * density
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        v = c * (z + 0.044715 * z * z * z)
        sig, rest = 1 / (1 + torch.exp(-v)), 1 / (1 + torch.exp(v))
        return sig + z * sig * rest * c * (1 + 3 * 0.044715 * z * z)
    sig, rest = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    return sig + z * sig * rest


def _values(q, scale):
    """fp32 rows from codes and scales."""
    return (_blocks(q.float()) * scale.unsqueeze(-1)).flatten(-2)[..., :q.shape[-1]]


def _run_plain(s):
    t, op, dtype = s["t"], s["op"], s["dtype"]
    if op == "norm":
        total = None
        v = t["x"].float()
        if s["residual"]:
            total = (v + t["residual"].float()).to(dtype)
            v = total.float()
        rstd = 1 / torch.sqrt((v * v).mean(1) + EPS)
        y = v * rstd.unsqueeze(1) * t["weight"].float()
        q, scale = _coded_rows(y)
        return {"q": q, "scale": scale, "total": total, "y": y.to(dtype) if s["dense"] else None,
                "rstd": rstd if s["save"] else None}
    if op == "norm_backward":
        v, r, dy = t["x"].float(), t["rstd"].unsqueeze(1), t["dy"].float()
        g = dy * t["weight"].float()
        dx = r * (g - v * (r * r) * (g * v).mean(1, keepdim=True))
        if s["through"]:
            dx = dx + t["dt"].float()
        return {"dx": dx.to(dtype), "dweight": (dy * v * r).sum(0)}
    if op.startswith("gated"):
        g, u = t["gu"].float().chunk(2, 1)
        if op == "gated":
            q, scale = _coded_rows(_act(s["act"], g) * u)
        else:
            dh = t["dh"].float()
            q, scale = _coded_rows(torch.cat([dh * u * _act_grad(s["act"], g),
                                              dh * _act(s["act"], g)], 1))
        return {"q": q, "scale": scale}
    w = t["codes"].float() * _spread(t["wscale"], s["N"], s["K"])
    if not op.endswith("backward"):
        w = w.transpose(-1, -2)
    x = _values(t["q"], t["scale"])
    if op.startswith("grouped"):
        row = torch.arange(s["T"], device=DEVICE)
        expert = torch.searchsorted(t["offsets"][1:], row, right=True)
        place = row - t["offsets"].long()[expert]
        padded = x.new_zeros(s["E"], s["most"], x.shape[1])
        padded[expert, place] = x
        y = torch.bmm(padded, w)[expert, place].to(dtype)
    else:
        y = (x @ w).to(dtype)
    return {"dx" if op.endswith("backward") else "y": y}


# ---------------------------------------------------------------------------
# the definition in 64 bits


def _exact_codes(v):
    """(v / scale before its rounding to e4m3, scales)."""
    q, scales = torch.empty_like(v), []
    for c in range(0, v.shape[1], BLOCK):
        part = v[:, c:c + BLOCK]
        scale = part.abs().max(1).values.clamp_min(FLOOR) / TOP
        q[:, c:c + BLOCK] = part / scale[:, None]
        scales.append(scale)
    return {"q": q, "scale": torch.stack(scales, 1)}


def _exact_act(name, z):
    """The activation and its derivative."""
    if name == "relu":
        return z.clamp_min(0.0), (z > 0).double()
    if name == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * torch.sigmoid(-z)
    if name == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(8.0 / math.pi)
    v = a * (z + 0.044715 * z ** 3)
    sig = torch.sigmoid(v)
    return z * sig, sig + z * sig * torch.sigmoid(-v) * a * (1.0 + 0.134145 * z ** 2)


def _exact_product(q, scale, codes, wscale, backward):
    """Block by block of the summed index."""
    n_out = codes.shape[1] if backward else codes.shape[0]
    total = torch.zeros(q.shape[0], n_out, dtype=torch.float64, device=q.device)
    spread = torch.arange(n_out, device=q.device) // BLOCK
    for b in range(scale.shape[1]):
        sl = slice(b * BLOCK, (b + 1) * BLOCK)
        w = codes[sl].double() if backward else codes[:, sl].double().t()
        s = (wscale[b] if backward else wscale[:, b]).double()
        total += (q[:, sl].double() @ w) * scale[:, b:b + 1].double() * s[spread]
    return total


def exact(case, seed):
    t = _inputs(case, seed)
    op, dtype = case["op"], TYPES[case["type"]]
    if op == "norm":
        v, total = t["x"].double(), None
        if case["residual"]:
            total = v + t["residual"].double()
            v = total.to(dtype).double()   # the norm is that of the stream as it is stored
        rstd = (torch.einsum("mk,mk->m", v, v) / case["K"] + EPS).rsqrt()
        y = torch.einsum("mk,m,k->mk", v, rstd, t["weight"].double())
        return dict(_exact_codes(y), total=total, y=y if case["dense"] else None,
                    rstd=rstd if case["save"] else None)
    if op == "norm_backward":
        v, r, dy, w = (t[k].double() for k in ("x", "rstd", "dy", "weight"))
        dot = torch.einsum("mk,mk,k->m", dy, v, w) / case["K"]
        dx = dy * w * r[:, None] - v * (dot * r ** 3)[:, None]
        if case["through"]:
            dx += t["dt"].double()
        return {"dx": dx, "dweight": torch.einsum("mk,mk,m->k", dy, v, r)}
    if op.startswith("gated"):
        F = case["F"]
        g, u = t["gu"][:, :F].double(), t["gu"][:, F:].double()
        f, df = _exact_act(case["act"], g)
        if op == "gated":
            return _exact_codes(f * u)
        dh = t["dh"].double()
        return _exact_codes(torch.cat([dh * u * df, dh * f], 1))
    backward = op.endswith("backward")
    name = "dx" if backward else "y"
    if op.startswith("linear"):
        return {name: _exact_product(t["q"], t["scale"], t["codes"], t["wscale"], backward)}
    at = t["offsets"].tolist()
    return {name: torch.cat([_exact_product(t["q"][a:b], t["scale"][a:b], t["codes"][e],
                                            t["wscale"][e], backward)
                             for e, (a, b) in enumerate(zip(at, at[1:])) if b > a])}


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]

    def coded(rows, cols):
        return rows * cols + 4 * rows * -(-cols // BLOCK)

    if op == "norm":
        M, K = case["M"], case["K"]
        size = 2 * M * K
        moved = size + 2 * K + coded(M, K)
        moved += 2 * size if case["residual"] else 0
        moved += size if case["dense"] else 0
        moved += 4 * M if case["save"] else 0
        return {"bytes": moved, "flops": 8 * M * K}
    if op == "norm_backward":
        M, K = case["M"], case["K"]
        arrays = 4 if case["through"] else 3
        return {"bytes": 2 * arrays * M * K + 4 * M + 6 * K, "flops": 10 * M * K}
    if op == "gated":
        M, F = case["M"], case["F"]
        return {"bytes": 4 * M * F + coded(M, F), "flops": 10 * M * F}
    if op == "gated_backward":
        M, F = case["M"], case["F"]
        return {"bytes": 6 * M * F + coded(M, 2 * F), "flops": 20 * M * F}
    rows, K, N = case.get("M", case.get("T")), case["K"], case["N"]
    matrices = case.get("active", 1)
    weights = matrices * (N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK))
    ends = 4 * (case["E"] + 1) if "E" in case else 0
    inner, outer = (N, K) if op.endswith("backward") else (K, N)
    return {"bytes": weights + ends + coded(rows, inner) + 2 * rows * outer,
            "flops": 2 * rows * N * K}
