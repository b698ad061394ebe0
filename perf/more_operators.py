"""Cases for the gated feed-forward layer and for products with group-scaled 4-bit weights.

Operators, and the entry points of dense_gemm_accelerator_gb300 that compute them:

  gated      H = act(X Wg^T + bg) * (X Wu^T + bu), W and the bias holding the gate's rows
             before the up projection's; where it is trained also the pre-activations
             P = X W^T + b that its gradients need: gated_forward
  backward   the gradients of X, W and the bias for H's gradient: gated_backward
  q4         Y = X W^T + b, W held as 4-bit codes with a scale (and a zero point) per group
             of 32, 64 or 128 values along K: q4_linear_forward
  q4_gated   the gated layer on such a weight: q4_gated_forward
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token through a served layer: the weight's bytes
        {"name": "gated 1 token", "op": "gated", "M": 1, "D": 4096, "F": 4096, "dtype": "bf16", "act": "silu", "bias": False, "save": False},
        # a few sequences decoding at once, odd in number, the larger weight
        {"name": "gated 13 tokens", "op": "gated", "M": 13, "D": 4096, "F": 8192, "dtype": "f16", "act": "gelu", "bias": True, "save": False},
        # a short prompt in fp32 at sizes that no tile divides, kept for its gradients
        {"name": "gated 509 f32", "op": "gated", "M": 509, "D": 515, "F": 1030, "dtype": "f32", "act": "gelu_tanh", "bias": True, "save": True},
        # the forward pass of a training step
        {"name": "gated 8192", "op": "gated", "M": 8192, "D": 4096, "F": 8192, "dtype": "bf16", "act": "silu", "bias": False, "save": True},
        # gradients of a small layer in fp32
        {"name": "backward 256 f32", "op": "backward", "M": 256, "D": 512, "F": 700, "dtype": "f32", "act": "silu", "bias": False},
        # ragged sizes with biases
        {"name": "backward 1000", "op": "backward", "M": 1000, "D": 1030, "F": 515, "dtype": "f16", "act": "gelu", "bias": True},
        # the largest: the gradients of a training step
        {"name": "backward 8192", "op": "backward", "M": 8192, "D": 4096, "F": 8192, "dtype": "bf16", "act": "silu", "bias": False},
        # one token through a projection: latency
        {"name": "q4 1 token", "op": "q4", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "group": 128, "zeros": True, "bias": False},
        # sequences decoding together, the smallest groups
        {"name": "q4 13 tokens", "op": "q4", "M": 13, "N": 8192, "K": 8192, "dtype": "f16", "group": 32, "zeros": False, "bias": True},
        # a prompt, an odd number of outputs
        {"name": "q4 300 tokens", "op": "q4", "M": 300, "N": 4099, "K": 4096, "dtype": "bf16", "group": 64, "zeros": True, "bias": False},
        # one token through a feed-forward block's gated part
        {"name": "q4 gated 1 token", "op": "q4_gated", "M": 1, "D": 4096, "F": 8192, "dtype": "bf16", "group": 128, "zeros": True, "act": "silu", "bias": False},
        # a few tokens, odd sizes, the last group part-filled
        {"name": "q4 gated 5 tokens", "op": "q4_gated", "M": 5, "D": 4093, "F": 4099, "dtype": "f16", "group": 64, "zeros": True, "act": "gelu_tanh", "bias": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "gated", "backward", "q4", "q4", "q4_gated"])
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
    if op == "q4":
        return {"op": op, "M": _log(rng, 1, 1024), "N": _log(rng, 256, 8192), "K": _log(rng, 256, 8192),
                "dtype": rng.choice(["bf16", "f16"]), "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "bias": rng.random() < 0.5}
    if op == "q4_gated":
        return {"op": op, "M": _log(rng, 1, 256), "D": _log(rng, 256, 8192), "F": _log(rng, 256, 8192),
                "dtype": rng.choice(["bf16", "f16"]), "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5,
                "act": act, "bias": rng.random() < 0.5}
    D, F = _log(rng, 256, 8192), _log(rng, 256, 8192)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "gated":  # from one token to a training step's
        M = min(_log(rng, 1, 8192), int(5e11 / (D * F)))
        return {"op": op, "M": M, "D": D, "F": F, "dtype": dtype, "act": act, "bias": rng.random() < 0.5, "save": rng.random() < 0.5}
    M = min(_log(rng, 32, 8192), int(2.5e11 / (D * F)))
    return {"op": op, "M": M, "D": D, "F": F, "dtype": dtype, "act": act, "bias": rng.random() < 0.5}


# ---- inputs -------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _activations(g, rows, cols, dtype):
    """Normal values whose columns differ in size, a few of them by much."""
    size = torch.exp(0.5 * _randn(g, cols))
    size[torch.rand(cols, device="cuda", generator=g) < 0.005] *= 10.0
    return (_randn(g, rows, cols) * size).to(dtype)


def _weight(g, rows, cols):
    return _randn(g, rows, cols) / math.sqrt(cols)


def _gradients(g, rows, cols, dtype):
    """Small values whose rows (tokens) differ in size; fp16 ones as a scaled loss gives them."""
    return (_randn(g, rows, cols) * torch.exp(_randn(g, rows, 1)) * (0.05 if dtype is torch.float16 else 1e-3)).to(dtype)


def _in_4_bits(w, group, zeros, dtype):
    """(codes, scales, zero points) of a weight's rows: two codes to a byte, the even value's
    in the low half, rows of whole 16 bytes; a scale and a zero point (None: 8) per group."""
    rows, cols = w.shape
    n = -(-cols // group)
    x = torch.nn.functional.pad(w, (0, n * group - cols)).reshape(rows, n, group)
    if zeros:
        lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        scale = ((hi - lo) / 15).to(dtype)
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (x.abs().amax(-1) / 7).to(dtype)
        zero = torch.full_like(scale, 8, dtype=torch.float32)
    code = torch.round(x / scale.float().unsqueeze(-1) + zero.unsqueeze(-1)).clamp(0, 15)
    code = code.to(torch.uint8).reshape(rows, -1)[:, :cols]
    code = torch.nn.functional.pad(code, (0, -cols % 32))
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), scale, zero.to(torch.uint8) if zeros else None


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DT[case["dtype"]]
    s = {"op": op, "act": case.get("act"), "save": case.get("save", False)}
    M = case["M"]
    K = case["K"] if op == "q4" else case["D"]
    N = case["N"] if op == "q4" else 2 * case["F"]
    s["X"] = _activations(g, M, K, dt)
    W = _weight(g, N, K)
    b = _randn(g, N).to(dt) if case["bias"] else None
    s["bias"] = b
    if op in ("q4", "q4_gated"):
        s["cols"], s["group"] = K, case["group"]
        s["codes"], s["scales"], s["zeros"] = _in_4_bits(W, case["group"], case["zeros"], dt)
        return s
    s["W"] = W.to(dt)
    if op == "backward":
        P = s["X"] @ s["W"].t()  # what the forward pass kept
        s["P"] = P if b is None else (P.float() + b.float()).to(dt)
        s["G"] = _gradients(g, M, case["F"], dt)
    return s


# ---- the plain form -------------------------------------------------------------


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g))
    return 1 / (1 + torch.exp(-g))


def _slope(g, act):
    """The activation's derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    if act == "relu":
        return (g > 0).to(g.dtype)
    s = 1 / (1 + torch.exp(-g))
    return s * (1 - s)


def _read(s):
    """The values that 4-bit codes, scales and zero points stand for."""
    codes, cols, group = s["codes"], s["cols"], s["group"]
    q = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :cols].float()
    scale = s["scales"].float().repeat_interleave(group, 1)[:, :cols]
    if s["zeros"] is None:
        return (q - 8) * scale
    return (q - s["zeros"].float().repeat_interleave(group, 1)[:, :cols]) * scale


def _plain(s):
    op, X, dt = s["op"], s["X"].float(), s["X"].dtype
    W = _read(s) if "codes" in s else s["W"].float()
    if op == "backward":
        gate, up = s["P"].float().chunk(2, 1)
        G = s["G"].float()
        dP = torch.cat([G * up * _slope(gate, s["act"]), G * _act(gate, s["act"])], 1)
        got = {"dX": (dP @ W).to(dt), "dW": (dP.t() @ X).to(dt)}
        return got if s["bias"] is None else {**got, "db": dP.sum(0)}
    P = X @ W.t()
    if s["bias"] is not None:
        P = P + s["bias"].float()
    if op == "q4":
        return P.to(dt)
    gate, up = P.chunk(2, 1)
    H = (_act(gate, s["act"]) * up).to(dt)
    return {"H": H, "P": P.to(dt)} if s["save"] else H


# ---- the framework's operators ----------------------------------------------------


def run(s):
    if not own:
        return _plain(s)
    import dense_gemm_accelerator_gb300 as dga
    op = s["op"]
    if op == "gated":
        if not s["save"]:
            return dga.gated_forward(s["X"], s["W"], s["bias"], activation=s["act"])
        H, P = dga.gated_forward(s["X"], s["W"], s["bias"], activation=s["act"], save=True)
        return {"H": H, "P": P}
    if op == "backward":
        dX, dW, db = dga.gated_backward(s["X"], s["W"], s["P"], s["G"], activation=s["act"], need_bias=s["bias"] is not None)
        return {"dX": dX, "dW": dW} if db is None else {"dX": dX, "dW": dW, "db": db}
    Q = dga.Q4Tensor(s["cols"], s["group"], s["codes"], s["scales"], s["zeros"])
    if op == "q4":
        return dga.q4_linear_forward(s["X"], Q, s["bias"])
    return dga.q4_gated_forward(s["X"], Q, s["bias"], activation=s["act"])


# ---- work -------------------------------------------------------------------------


def work(case):
    op, M = case["op"], case["M"]
    e = 4 if case["dtype"] == "f32" else 2
    if op in ("q4", "q4_gated"):
        K = case["K"] if op == "q4" else case["D"]
        N = case["N"] if op == "q4" else 2 * case["F"]
        out = N if op == "q4" else case["F"]
        groups = -(-K // case["group"])
        held = N * (K / 2 + groups * (3 if case["zeros"] else 2))
        return {"bytes": held + 2 * (M * K + M * out + (N if case["bias"] else 0)), "flops": 2.0 * M * N * K}
    D, F = case["D"], case["F"]
    if op == "gated":
        outputs = M * F * (3 if case["save"] else 1)
        return {"bytes": e * (M * D + 2 * F * D + outputs + (2 * F if case["bias"] else 0)), "flops": 4.0 * M * F * D}
    # X, W, P and G in; dX, dW and (fp32) db out
    return {"bytes": e * (2 * M * D + 4 * F * D + 3 * M * F) + (8 * F if case["bias"] else 0), "flops": 8.0 * M * F * D}


# ---- the definition in 64 bits ------------------------------------------------------


def _exact_act(x, act):
    """(value, derivative) in fp64."""
    if act == "relu":
        return torch.clamp(x, min=0.0), torch.heaviside(x, torch.zeros_like(x))
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * torch.exp(-x.square() / 2) / math.sqrt(math.tau)
    if act == "gelu_tanh":  # (1 + tanh v) / 2 is the logistic function of 2 v
        v = math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3)
        p = torch.sigmoid(v)
        return x * p, p + x * p * torch.sigmoid(-v) * math.sqrt(8 / math.pi) * (1 + 0.134145 * x.square())
    p, q = torch.sigmoid(x), torch.sigmoid(-x)
    if act == "silu":
        return x * p, p + x * p * q
    return p, p * q


def exact(case, seed):
    s = prepare(case, seed)
    X = s["X"].double()
    if "codes" in s:
        low, high = (s["codes"].long() % 16).double(), (s["codes"].long() // 16).double()
        q = torch.empty(low.shape[0], 2 * low.shape[1], dtype=torch.float64, device=low.device)
        q[:, 0::2], q[:, 1::2] = low, high
        at = torch.arange(s["cols"], device=q.device) // s["group"]
        zero = 8.0 if s["zeros"] is None else s["zeros"].double()[:, at]
        W = (q[:, :s["cols"]] - zero) * s["scales"].double()[:, at]
    else:
        W = s["W"].double()
    if case["op"] == "backward":
        F = case["F"]
        P, G = s["P"].double(), s["G"].double()
        value, slope = _exact_act(P[:, :F], s["act"])
        dgate, dup = G * P[:, F:] * slope, G * value
        got = {"dX": torch.addmm(dgate @ W[:F], dup, W[F:]), "dW": torch.cat([dgate.mT @ X, dup.mT @ X])}
        if s["bias"] is not None:
            got["db"] = torch.cat([dgate.sum(0), dup.sum(0)])
        return got
    P = torch.einsum("mk,nk->mn", X, W)
    if s["bias"] is not None:
        P += s["bias"].double()
    if case["op"] == "q4":
        return P
    F = case["F"]
    H = _exact_act(P[:, :F], s["act"])[0] * P[:, F:]
    return {"H": H, "P": P} if s["save"] else H
