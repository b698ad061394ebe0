"""Plain 64-bit forms of the gated layer, its gradients and the group-scaled
4-bit weights, with bounds on what a kernel that sums in fp32 may be off by.

Bounds.  A sum of n products taken in fp32, in any order, is off by at most
n 2^-24 (1 + small) of the sum of the products' magnitudes; SUM allows 16 more
for the pieces' own sums.  A result rounded to a type is off by eps / 2 of its
value, or half a step of the type's least numbers (HALF, TINY).  An activation
evaluated in fp32 is allowed 2^-17 of max(1, |g|) (the hardware's exponential
and reciprocal are within 2^-20 of their value here); its slope's magnitude is at
most 1.13 for every activation of these, which carries an error of g to act(g)."""
import math

import torch

ACTS = ["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
# half a step of the least numbers; fp32 results below the normal range may be flushed
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
ACT_ERR = 2.0 ** -17


def act(g, name):
    if name == "relu":
        return torch.where(g > 0, g, torch.where(g == g, torch.zeros_like(g), g))
    if name == "gelu":
        return g * torch.special.erfc(-g / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    s = 1 / (1 + torch.exp(-g))
    return g * s if name == "silu" else s


def slope(g, name):
    if name == "relu":
        return (g > 0).to(g.dtype)
    if name == "gelu":
        return torch.special.erfc(-g / math.sqrt(2)) / 2 + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (g + 0.044715 * g ** 3)))
        return s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)
    s = 1 / (1 + torch.exp(-g))
    return s * (1 + g * (1 - s)) if name == "silu" else s * (1 - s)


def sum_error(n):
    return (n + 16) * 2.0 ** -24


def rounding(v, dtype):
    return HALF[dtype] * v.abs() + TINY[dtype]


def product(X, W, bias=None):
    """(X W^T + bias, how far fp32 sums may be off) in fp64."""
    X, W = X.double(), W.double()
    v = X @ W.t()
    off = sum_error(X.shape[1]) * (X.abs() @ W.abs().t())
    if bias is not None:
        v = v + bias.double()
        off = off + 2.0 ** -23 * (v.abs() + bias.double().abs())
    return v, off


def gated_of(P, off, name, dtype):
    """(H, its bound) from pre-activations and how far they are off."""
    F = P.shape[1] // 2
    g, u, dg, du = P[:, :F], P[:, F:], off[:, :F], off[:, F:]
    a = act(g, name)
    H = a * u
    ea = 1.13 * dg + ACT_ERR * torch.clamp(g.abs(), min=1.0)
    return H, (ea * (u.abs() + du) + a.abs() * du) * (1 + 2.0 ** -8) + rounding(H, dtype) + 2.0 ** -23 * H.abs()


def gated(X, W, bias, name):
    """H, P and their bounds."""
    P, off = product(X, W, bias)
    H, eh = gated_of(P, off, name, X.dtype)
    return H, eh, P, off * (1 + HALF[X.dtype]) + rounding(P, X.dtype)


def gated_grads(X, W, P, G, name):
    """{name: (value, bound)} of dX, dW, db."""
    dtype = X.dtype
    X, W, P, G = X.double(), W.double(), P.double(), G.double()
    F = G.shape[1]
    g, u = P[:, :F], P[:, F:]
    a, s = act(g, name), slope(g, name)
    dP = torch.cat([G * u * s, G * a], 1)
    big = torch.clamp(g.abs(), min=1.0)
    e = torch.cat([(G * u).abs() * ACT_ERR * big, G.abs() * ACT_ERR * big], 1) + 2.0 ** -22 * dP.abs()
    er = e + rounding(dP, dtype) if dtype != torch.float32 else e
    out = {}
    for key, L, R, EL in (("dX", dP, W, er), ("dW", dP.t(), X, er.t())):
        v = L @ R
        off = EL @ R.abs() + sum_error(L.shape[1]) * (L.abs() @ R.abs())
        out[key] = (v, off * (1 + 2.0 ** -8) + rounding(v, dtype))
    out["db"] = (dP.sum(0), e.sum(0) + sum_error(P.shape[0]) * dP.abs().sum(0) + TINY[torch.float32])
    return out


def within(got, want, bound, what=""):
    got = got.double()
    err = (got - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / bound)[bad].max()), bad.nonzero()[0].tolist())


# ---- 4-bit weights ------------------------------------------------------------------


def q4_quantize(W, group, zeros, scale_dtype):
    """(codes one to a value, scales, zero points) by the definition, W on the CPU; each
    fp32 operation correctly rounded, as PyTorch's CPU ones are."""
    rows, cols = W.shape
    n = -(-cols // group)
    w = torch.zeros(rows, n * group)
    w[:, :cols] = W.float()
    w = w.view(rows, n, group)
    lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
    fine = torch.isfinite(w).all(-1)
    s = ((hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7).to(scale_dtype)
    fine = fine & torch.isfinite(s)
    sf = s.float()
    use = fine & (sf > 0)
    one = torch.where(use, sf, torch.ones_like(sf))
    z = torch.where(use, torch.round(-lo / one).clamp(0, 15), torch.zeros_like(sf)) if zeros else torch.full_like(sf, 8)
    q = torch.round(w / one.unsqueeze(-1) + z.unsqueeze(-1)).clamp(0, 15)
    q = torch.where(use.unsqueeze(-1), q, z.unsqueeze(-1)).view(rows, -1)[:, :cols]
    s = torch.where(fine, s, torch.full_like(s, math.nan))
    return q.to(torch.uint8), s, z.to(torch.uint8)


def q4_unpack(codes, cols):
    return torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)[:, :cols]


def q4_values(codes, scales, zeros, cols, group):
    """The values in fp64."""
    q = q4_unpack(codes, cols).double()
    s = scales.double().repeat_interleave(group, 1)[:, :cols]
    z = 8.0 if zeros is None else (zeros & 15).double().repeat_interleave(group, 1)[:, :cols]
    return (q - z) * s
