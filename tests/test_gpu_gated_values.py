"""The gates' values and slopes one by one, against fp64 relative to themselves: products
of one term each (K = 1, X = 1, up = 1, G = 1), so that a result is act(g) rounded once and
db, which is fp32 in every type, the slope.

Bounds.  In units of STEP = 2^-23: the CUDA guide gives the hardware's exponential
2 + 1.173 |x| and its division 2, and the library's exponential 2, and its normal
distribution 5; the fitted Phi of the 16-bit kernels is 7e-7 off by its fit and the
exponent x^2 = g^2 / 2 loses five halves of a step of itself; every other operation half a
step.  The logistic function so is 8 + 1.2 |x| off (16-bit kernels) or 8 (fp32), and for
gelu_tanh the argument v of 4 roundings adds 2 |v|."""
import math

import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import gated_reference as ref

STEP = 2.0 ** -23
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def gates(dtype, count):
    """`count` gates: -13 to 20, where fp32 runs out of the exponential, and far ones."""
    far = torch.tensor([-87.25, -87.5, -88.0, -88.5, -60.0, -40.0, -30.0, 30.0, 60.0, 88.5, 200.0, 6e4, 0.0, 2.0 ** -20, -2.0 ** -20])
    return torch.cat([torch.linspace(-13, 20, count - far.numel()), far]).to(dtype)


def exact(g, name):
    """(value, its bound, slope, its bound) relative parts for the 16-bit kernels (fast) and fp32."""
    g = g.double()
    out = {}
    for fast in (False, True):
        if name == "relu":
            zero = torch.zeros_like(g)
            out[fast] = (g.clamp(min=0), zero, (g > 0).double(), zero)
        elif name == "gelu":
            c = torch.special.erfc(-g / math.sqrt(2)) / 2
            phi = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
            x = g * g / 2
            rc = (1e-6 + (5 + 2.5 * x) * STEP) if fast else torch.full_like(g, 8 * STEP)
            # the value for g > 0 is 1 - (the other tail), whose error is then one of 1
            ec = torch.maximum(rc * c, rc * (1 - c)) if fast else rc * c
            rp = (6 + (3.2 if fast else 2) * x) * STEP
            out[fast] = (g * c, ec * g.abs() + 2 * STEP * (g * c).abs(), c + g * phi, ec + rp * (g * phi).abs() + 2 * STEP * (c + g * phi).abs())
        else:
            v = g if name != "gelu_tanh" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
            s, t = torch.sigmoid(v), torch.sigmoid(-v)
            r = (8 + (1.2 * v.abs() if fast else 0) + (2 * v.abs() if name == "gelu_tanh" else 0)) * STEP
            # the larger of s and t is 1 less the smaller: off by what that is off by
            small = torch.minimum(s, t)
            es, et = (torch.where(w == small, r * w, 4 * STEP + r * small) for w in (s, t))
            st, est = s * t, es * t + et * s + STEP * s * t
            if name == "sigmoid":
                out[fast] = (s, es, st, est)
            else:
                d = torch.ones_like(g) if name == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
                far = st == 0  # (0 times a d that may have passed any range)
                slope = s + torch.where(far, torch.zeros_like(g), g * st * d)
                e = es + torch.where(far, torch.zeros_like(g), g.abs() * d * est + 4 * STEP * (g * st * d).abs()) + STEP * slope.abs()
                out[fast] = (g * s, es * g.abs() + STEP * (g * s).abs(), slope, e)
    return out


def check(got, want, bound, dtype, what):
    """Within the bound, a rounding to dtype, and fp32's or the type's least numbers."""
    ref.within(got, want, bound + ref.HALF[dtype] * (want.abs() + bound) + ref.TINY[dtype], what)


# ---- the bounds themselves, on the CPU ------------------------------------------------


@pytest.mark.parametrize("name", ref.ACTS)
def test_the_bounds_hold_for_correctly_rounded_steps_and_see_a_difference(name):
    """Elementary functions rounded from fp64 stay within the bounds; a slope by 1 - s does not."""
    g = gates(torch.float32, 2000)
    value, ev, slope, es = exact(g, name)[False]
    check(ref.act(g.double(), name).nan_to_num(0.0).float(), value, ev, torch.float32, name)
    check(slope.float(), slope, es, torch.float32, name)
    if name == "sigmoid":
        e = torch.exp(-g.double()).float()
        s = 1 / (1 + e)
        with pytest.raises(AssertionError):
            check(s * (1 - s), slope, es, torch.float32, name)
        low = g < 0  # where 1 - s loses nothing
        check((s * (1 - s))[low], slope[low], es[low], torch.float32, name)


# ---- the kernels ----------------------------------------------------------------------


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M,F", [(1, 2048), (3, 771), (40, 2048), (40, 771)])
def test_values_and_slopes(M, F, name, dtype):
    g = gates(dtype, F).cuda()
    one = torch.ones(F, dtype=dtype, device="cuda")
    X = torch.ones(M, 1, dtype=dtype, device="cuda")
    W = torch.cat([g, one])[:, None].contiguous()
    H, P = dga.gated_forward(X, W, activation=name, save=True)
    assert torch.equal(P, W[:, 0].expand(M, 2 * F))
    value, ev, slope, es = exact(g, name)[dtype != torch.float32]
    check(H, value.expand(M, F), ev.expand(M, F), dtype, "value")
    # one row, so that db is the slope (and the value) as computed
    db = dga.gated_backward(X[:1], W, P[:1], one[None], activation=name, need_bias=True)[2]
    check(db[:F], slope, es, torch.float32, "slope")
    check(db[F:], value, ev, torch.float32, "value as up's gradient")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("M", [1, 40, 100, 600])
def test_values_on_4_bit_weights(M, name, dtype):
    """g as a group's scale times the code 9 less 8."""
    F = 771
    g = gates(dtype, F).cuda()
    codes = torch.zeros(2 * F, 16, dtype=torch.uint8, device="cuda")
    codes[:, 0] = 9
    Q = dga.Q4Tensor(1, 32, codes, torch.cat([g, torch.ones_like(g)])[:, None].contiguous())
    H = dga.q4_gated_forward(torch.ones(M, 1, dtype=dtype, device="cuda"), Q, activation=name)
    value, ev = exact(g, name)[True][:2]
    check(H, value.expand(M, F), ev.expand(M, F), dtype, name)
