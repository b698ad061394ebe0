"""Cases for the microscaled 4-bit operators and the orthogonalised update.

Operators, and the entry points of dense_gemm_accelerator_gb300 that compute them:

  round_trip   a matrix to 4-bit codes and block scales (its rows, or its
               columns with transpose=True) and back to values:
               mx_quantize, mx_dequantize
  linear       the fully-connected layer on a 4-bit weight, quantising the
               activations on the way: mx_linear_forward
  product      C = alpha A B^T of two matrices already in 4 bits: mx_gemm
  backward     the layer's gradients with 4-bit products: mx_linear_backward
  orthogonal   an update's Newton-Schulz orthogonalisation: orthogonalize

Formats: "mx" is E2M1 codes with one E8M0 scale per 32 values, "nv" E2M1 codes
with one E4M3 scale per 16 values and one fp32 factor per tensor.
"""
import math

import torch

own = False

# the quintic of the Newton-Schulz iteration: X <- a X + (b A + c A^2) X, A = X X^T
QUINTIC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token through a square layer: latency, the weight's bytes
        {"name": "linear 1 token", "op": "linear", "fmt": "mx", "T": 1, "N": 4096, "K": 4096, "dtype": "bf16", "bias": False},
        # a few sequences decoding at once, odd in number, the larger weight
        {"name": "linear 13 tokens", "op": "linear", "fmt": "nv", "T": 13, "N": 8192, "K": 8192, "dtype": "bf16", "bias": True},
        # a short prompt: between the bandwidth and the tensor cores' rate
        {"name": "linear 509 tokens", "op": "linear", "fmt": "mx", "T": 509, "N": 8192, "K": 4096, "dtype": "f16", "bias": True},
        # the largest product, operands already quantised
        {"name": "product 8192", "op": "product", "fmt": "mx", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # sizes that no tile divides, fp32 output
        {"name": "product ragged", "op": "product", "fmt": "nv", "M": 4093, "N": 4099, "K": 4097, "out": "f32"},
        # a few rows of cached values written and read back
        {"name": "round trip 37 rows", "op": "round_trip", "fmt": "nv", "rows": 37, "cols": 1000, "dtype": "f32", "transpose": False},
        # a large activation along its other axis, as a weight gradient needs it
        {"name": "round trip 8192 transposed", "op": "round_trip", "fmt": "mx", "rows": 8192, "cols": 8192, "dtype": "bf16", "transpose": True},
        # one layer's gradients
        {"name": "backward 4096", "op": "backward", "fmt": "mx", "T": 4096, "N": 4096, "K": 4096, "dtype": "bf16"},
        # the update of a small projection: launches and latency
        {"name": "orthogonal 256", "op": "orthogonal", "batch": 1, "m": 256, "n": 256, "dtype": "f32"},
        # one shape of every layer at once, odd sizes, more rows than columns
        {"name": "orthogonal 12 x 1030 x 515", "op": "orthogonal", "batch": 12, "m": 1030, "n": 515, "dtype": "bf16"},
        # a wide layer held in fp32
        {"name": "orthogonal 1000 x 4099 f32", "op": "orthogonal", "batch": 1, "m": 1000, "n": 4099, "dtype": "f32"},
        # the largest update
        {"name": "orthogonal 4096", "op": "orthogonal", "batch": 1, "m": 4096, "n": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "product", "round_trip", "backward", "orthogonal", "orthogonal"])
    fmt = rng.choice(["mx", "nv"])
    if op == "linear":
        return {"op": op, "fmt": fmt, "T": _log(rng, 1, 2048), "N": _log(rng, 500, 8192), "K": _log(rng, 500, 8192),
                "dtype": rng.choice(["bf16", "f16"]), "bias": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "fmt": fmt, "M": _log(rng, 100, 8192), "N": _log(rng, 500, 8192), "K": _log(rng, 500, 8192),
                "out": rng.choice(["bf16", "f32"])}
    if op == "round_trip":
        return {"op": op, "fmt": fmt, "rows": _log(rng, 16, 8192), "cols": _log(rng, 100, 8192),
                "dtype": rng.choice(["bf16", "f16", "f32"]), "transpose": rng.random() < 0.5}
    if op == "backward":
        return {"op": op, "fmt": fmt, "T": _log(rng, 64, 4096), "N": _log(rng, 200, 4096), "K": _log(rng, 200, 4096),
                "dtype": "bf16"}
    m, n = _log(rng, 48, 3000), _log(rng, 48, 3000)
    return {"op": op, "batch": max(1, min(_log(rng, 1, 16), int(1.2e7 / (m * n)))), "m": m, "n": n,
            "dtype": rng.choice(["bf16", "f32"])}


# ---- inputs -------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _activations(g, rows, cols, dtype):
    """Normal values whose columns differ in size, a few of them by much."""
    size = torch.exp(0.5 * _randn(g, cols))
    size[torch.rand(cols, device="cuda", generator=g) < 0.005] *= 20.0
    return (_randn(g, rows, cols) * size).to(dtype)


def _gradients(g, rows, cols, dtype):
    """Small values whose rows (tokens) differ in size."""
    return (_randn(g, rows, cols) * torch.exp(_randn(g, rows, 1)) * 1e-3).to(dtype)


def _factor(x, fmt):
    """The tensor's factor, which brings its largest block scale to the upper half of E4M3's
    range; a power of two, so that dividing by it rounds nothing."""
    if fmt != "nv":
        return None
    r = (x.abs().amax().float() / 2688.0).reshape(1)
    return r / torch.frexp(r).mantissa


def prepare(case, seed):
    g = _gen(seed)
    op, fmt = case["op"], case.get("fmt")
    s = {"op": op, "fmt": fmt}
    if op == "orthogonal":
        shape = (case["batch"], case["m"], case["n"])
        k = max(1, min(case["m"], case["n"]) // 32)  # momentum: a few directions over noise
        s["G"] = (1e-3 * (_randn(g, *shape) + 0.5 * _randn(g, shape[0], shape[1], k) @ _randn(g, shape[0], k, shape[2]))).to(DT[case["dtype"]])
        return s
    if op == "round_trip":
        s["X"] = _activations(g, case["rows"], case["cols"], DT[case["dtype"]])
        s["gX"] = _factor(s["X"], fmt)
        s["transpose"] = case["transpose"]
        return s
    if op == "backward":
        dt = DT[case["dtype"]]
        s["X"] = _activations(g, case["T"], case["K"], dt)
        s["W"] = (_randn(g, case["N"], case["K"]) / math.sqrt(case["K"])).to(dt)
        s["G"] = _gradients(g, case["T"], case["N"], dt)
        s["gX"], s["gW"], s["gG"] = (_factor(s[k], fmt) for k in "XWG")
        return s
    if op == "linear":
        dt = DT[case["dtype"]]
        s["X"] = _activations(g, case["T"], case["K"], dt)
        W = (_randn(g, case["N"], case["K"]) / math.sqrt(case["K"])).to(dt)
        s["bias"] = _randn(g, case["N"]).to(dt) if case["bias"] else None
        s["gX"], s["gW"] = _factor(s["X"], fmt), _factor(W, fmt)
        s["W"] = _held(W, fmt, s["gW"])
        return s
    A = _activations(g, case["M"], case["K"], torch.bfloat16)
    B = (_randn(g, case["N"], case["K"]) / math.sqrt(case["K"])).bfloat16()
    s["gA"], s["gB"] = _factor(A, fmt), _factor(B, fmt)
    s["A"], s["B"] = _held(A, fmt, s["gA"]), _held(B, fmt, s["gB"])
    s["out"] = case["out"]
    return s


def _held(x, fmt, factor):
    """A matrix in 4 bits as a program keeps it: the framework's handle, or codes (one per
    byte, sign in bit 3) and block scales."""
    if own:
        import dense_gemm_accelerator_gb300 as dga
        return dga.mx_quantize(x, _format(dga, fmt), tensor_scale=factor)
    v, scale = _quantise(x, fmt, factor)
    a = v.abs()  # E2M1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 are codes 0 to 7
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    return (code + 8 * (v < 0).to(torch.uint8), scale, x.shape[1])


# ---- the plain form -------------------------------------------------------------

_LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _quantise(x, fmt, factor):
    """(values on the E2M1 grid, block scales) of the rows of x, padded to whole blocks."""
    x = x.float()
    block = 32 if fmt == "mx" else 16
    rows, cols = x.shape
    n = -(-cols // block)
    x = torch.nn.functional.pad(x, (0, n * block - cols)).reshape(rows, n, block)
    amax = x.abs().amax(-1)
    if fmt == "mx":
        m, e = torch.frexp(amax)  # amax = m 2^e with m in [1/2, 1): floor(log2 amax) = e - 1
        scale = torch.where((amax > 0) & (e > -124), amax / (8.0 * m), torch.full_like(amax, 2.0 ** -127))
        unit = scale
    else:
        scale = torch.clamp(amax / (6.0 * factor), max=448.0).to(torch.float8_e4m3fn).float()
        unit = scale * factor
    t = torch.where(unit.unsqueeze(-1) > 0, x / unit.unsqueeze(-1), torch.zeros_like(x))
    a = t.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.clamp(torch.round(a / step) * step, max=6.0)
    return torch.where(t < 0, -v, v).reshape(rows, n * block), scale


def _values(v, scale, cols, factor):
    """What values on the E2M1 grid and block scales stand for."""
    rows, n = scale.shape
    unit = scale if factor is None else scale * factor
    return (v.reshape(rows, n, -1) * unit.unsqueeze(-1)).reshape(rows, -1)[:, :cols]


def _near(x, fmt, factor):
    """x rounded to 4 bits along its rows."""
    return _values(*_quantise(x, fmt, factor), x.shape[1], factor)


def _read(held, factor):
    code, scale, cols = held
    v = _LEVELS.to(code.device)[(code & 7).long()]
    return _values(torch.where(code >= 8, -v, v), scale, cols, factor)


def _plain(s):
    op, fmt = s["op"], s["fmt"]
    if op == "round_trip":
        X = s["X"].t() if s["transpose"] else s["X"]
        return _near(X, fmt, s["gX"])
    if op == "linear":
        y = _near(s["X"], fmt, s["gX"]) @ _read(s["W"], s["gW"]).t()
        return (y if s["bias"] is None else y + s["bias"].float()).to(s["X"].dtype)
    if op == "product":
        return (_read(s["A"], s["gA"]) @ _read(s["B"], s["gB"]).t()).to(DT[s["out"]])
    if op == "backward":
        X, W, G = s["X"], s["W"], s["G"]
        dX = _near(G, fmt, s["gG"]) @ _near(W.t(), fmt, s["gW"]).t()
        dW = _near(G.t(), fmt, s["gG"]) @ _near(X.t(), fmt, s["gX"]).t()
        return {"dX": dX.to(G.dtype), "dW": dW.to(G.dtype), "db": G.float().sum(0)}
    a, b, c = QUINTIC
    X = s["G"].float()
    tall = X.shape[1] > X.shape[2]
    if tall:
        X = X.transpose(1, 2)
    X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(5):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.transpose(1, 2) if tall else X).to(s["G"].dtype)


# ---- the framework's operators ----------------------------------------------------


def _format(dga, fmt):
    return dga.MXFP4 if fmt == "mx" else dga.NVFP4


def run(s):
    if not own:
        return _plain(s)
    import dense_gemm_accelerator_gb300 as dga
    op = s["op"]
    if op == "round_trip":
        return dga.mx_dequantize(dga.mx_quantize(s["X"], _format(dga, s["fmt"]), transpose=s["transpose"], tensor_scale=s["gX"]))
    if op == "linear":
        return dga.mx_linear_forward(s["X"], s["W"], s["bias"], tensor_scale=s["gX"])
    if op == "product":
        return dga.mx_gemm(s["A"], s["B"], out_dtype=dga.BF16 if s["out"] == "bf16" else dga.F32)
    if op == "backward":
        dX, dW, db = dga.mx_linear_backward(s["X"], s["W"], s["G"], _format(dga, s["fmt"]), tensor_scales=(s["gX"], s["gW"], s["gG"]))
        return {"dX": dX, "dW": dW, "db": db}
    return dga.orthogonalize(s["G"], steps=5, coefficients=QUINTIC, eps=EPS)


# ---- work -------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "orthogonal":
        m, n = sorted((case["m"], case["n"]))
        e = case["batch"] * m * n * (4 if case["dtype"] == "f32" else 2)
        # X X^T and A^2 are symmetric: half of their entries
        return {"bytes": 2 * e, "flops": case["batch"] * 5 * (3.0 * m * m * n + 1.0 * m * m * m)}
    held = 0.5 + (1 / 32 if case["fmt"] == "mx" else 1 / 16)  # bytes of a 4-bit value
    if op == "round_trip":
        n = case["rows"] * case["cols"]
        # read, written in 4 bits, read again, written as fp32 values
        return {"bytes": n * ((4 if case["dtype"] == "f32" else 2) + 2 * held + 4), "flops": 0}
    if op == "linear":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K * 2 + N * K * held + T * N * 2, "flops": 2.0 * T * N * K}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * held + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2.0 * M * N * K}
    T, N, K = case["T"], case["N"], case["K"]
    return {"bytes": 2 * (T * K + N * K + T * N) + 2 * (T * K + N * K) + 4 * N, "flops": 4.0 * T * N * K}


# ---- the definition in 64 bits ------------------------------------------------------


def _binade(x, least, most):
    """2^floor(log2 x) in fp64, read from its bits and held to 2^least .. 2^most."""
    e = (x.view(torch.int64) >> 52) - 1023
    return (((torch.clamp(e, least, most)) + 1023) << 52).view(torch.float64)


def _exact_near(x, fmt, factor):
    """x (fp64) rounded to 4 bits along its rows, by the midpoints between E2M1's levels."""
    block = 32 if fmt == "mx" else 16
    rows, cols = x.shape
    pad = -cols % block
    b = torch.cat([x, x.new_zeros(rows, pad)], 1).view(rows, -1, block)
    top = b.abs().max(-1, keepdim=True).values
    if fmt == "mx":
        unit = _binade(top, -125, 127) / 4
    else:
        f = factor.double()
        r = torch.clamp(top / (6 * f), max=448.0)
        quantum = _binade(r, -6, 8) / 8
        unit = torch.round(r / quantum) * quantum * f
    t = torch.where(unit > 0, b / torch.where(unit > 0, unit, torch.ones_like(unit)), torch.zeros_like(b))
    a, q = t.abs(), torch.zeros_like(t)
    for level, mid, even in ((0.5, 0.25, False), (1.0, 0.75, True), (1.5, 1.25, False), (2.0, 1.75, True),
                             (3.0, 2.5, False), (4.0, 3.5, True), (6.0, 5.0, False)):
        q = torch.where((a >= mid) if even else (a > mid), torch.full_like(q, level), q)
    return (torch.sign(t) * q * unit).reshape(rows, -1)[:, :cols]


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    op, fmt = s["op"], s["fmt"]
    if op == "orthogonal":
        a, b, c = QUINTIC
        X = s["G"].double()
        wide = X if X.shape[1] <= X.shape[2] else X.mT
        U = wide / (torch.linalg.vector_norm(wide, dim=(1, 2), keepdim=True) + EPS)
        for _ in range(5):
            S = torch.bmm(U, U.mT)
            U = a * U + b * torch.bmm(S, U) + c * torch.bmm(S, torch.bmm(S, U))
        return U if wide is X else U.mT.contiguous()
    if op == "round_trip":
        X = s["X"].double()
        return _exact_near(X.t() if s["transpose"] else X, fmt, s["gX"])
    if op == "backward":
        X, W, G = (s[k].double() for k in "XWG")
        n = lambda t, f: _exact_near(t, fmt, f)  # noqa: E731
        return {"dX": n(G, s["gG"]) @ n(W.t(), s["gW"]).t(), "dW": n(G.t(), s["gG"]) @ n(X.t(), s["gX"]).t(),
                "db": G.sum(0)}
    if op == "linear":
        y = torch.einsum("tk,nk->tn", _exact_near(s["X"].double(), fmt, s["gX"]), _exact_held(s["W"], s["gW"]))
        return y if s["bias"] is None else y + s["bias"].double()
    return torch.einsum("mk,nk->mn", _exact_held(s["A"], s["gA"]), _exact_held(s["B"], s["gB"]))


def _exact_held(held, factor):
    """The fp64 values of codes and scales, from the E2M1 encoding's bits."""
    code, scale, cols = held
    c = code.long()
    e, man = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * man, (1 + 0.5 * man) * torch.exp2((e - 1).double()))
    v = torch.where((c >> 3) & 1 == 1, -v, v)
    unit = scale.double() if factor is None else scale.double() * factor.double()
    return (v.view(scale.shape[0], scale.shape[1], -1) * unit.unsqueeze(2)).flatten(1)[:, :cols]
