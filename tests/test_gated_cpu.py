"""The gated layer's and the group-scaled 4-bit entry points without a GPU:
argument errors (reported before the device is touched), sizes, and the test
reference by hand."""
import math

import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from dense_gemm_accelerator_gb300 import build as dga_build
from dense_gemm_accelerator_gb300 import inputs as gen
from tests import gated_reference as ref

P = [0x100000000 * i for i in range(1, 14)]  # never dereferenced
BIG = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def lib():
    dga_build.build()
    return dga.lib()


def _gated(**over):
    a = dict(dtype=gen.BF16, act=0, M=4, F=8, K=16, X=P[0], ldx=16, W=P[1], ldw=16, bias=None, H=P[2], ldh=8, P=None, ldp=0,
             workspace=P[3], workspace_bytes=1 << 24, stream=None)
    a.update(over)
    return dga.dga_gated(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(dtype=gen.I8), 1), (dict(dtype=gen.TF32), 1), (dict(act=5), 1), (dict(act=-1), 1),
    (dict(M=-1), -3), (dict(M=BIG), -3), (dict(F=-1), -4), (dict(F=BIG), -4), (dict(K=-1), -5),
    (dict(X=None), -6), (dict(X=P[0] + 1), -6), (dict(ldx=15), -7), (dict(W=None), -8), (dict(ldw=15), -9), (dict(bias=P[4] + 1), -10),
    (dict(H=None), -11), (dict(H=P[2] + 1), -11), (dict(ldh=7), -12), (dict(P=P[5] + 1, ldp=16), -13), (dict(P=P[5], ldp=15), -14),
    (dict(workspace=None), -15), (dict(workspace=P[3] + 8), -15),
    (dict(H=P[0]), 6), (dict(H=P[1] + 32), 6), (dict(P=P[2] + 2, ldp=16), 6), (dict(bias=P[2]), 6), (dict(workspace=P[1], dtype=gen.F32), 6),
    (dict(M=0, X=None, W=None, H=None), 0), (dict(F=0, W=None, H=None), 0)])
def test_gated_arguments(over, code):
    assert _gated(M=over.get("M", 40), **{k: v for k, v in over.items() if k != "M"}) == code


def _backward(**over):
    a = dict(dtype=gen.F16, act=1, M=40, F=8, K=16, X=P[0], ldx=16, W=P[1], ldw=16, P=P[2], ldp=16, G=P[3], ldg=8, dX=P[4], lddx=16,
             dW=P[5], lddw=16, db=P[6], workspace=P[7], workspace_bytes=1 << 24, stream=None)
    a.update(over)
    return dga.dga_gated_backward(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(dtype=gen.I32), 1), (dict(act=9), 1), (dict(M=BIG), -3), (dict(F=-1), -4), (dict(K=BIG), -5),
    (dict(X=None), -6), (dict(ldx=3), -7), (dict(W=None), -8), (dict(ldw=3), -9), (dict(P=None), -10), (dict(ldp=15), -11),
    (dict(G=None), -12), (dict(ldg=7), -13), (dict(dX=P[4] + 1), -14), (dict(lddx=15), -15), (dict(dW=P[5] + 1), -16), (dict(lddw=15), -17),
    (dict(db=P[6] + 2), -18), (dict(workspace=None), -19), (dict(workspace=P[7] + 16), -19), (dict(workspace_bytes=64), 5),
    (dict(dX=P[5]), 6), (dict(dW=P[1]), 6), (dict(dX=P[3]), 6), (dict(db=P[2]), 6), (dict(workspace=P[0]), 6)])
def test_backward_arguments(over, code):
    assert _backward(**over) == code


def _linear(**over):
    a = dict(dtype=gen.BF16, M=40, N=8, K=64, group=32, X=P[0], ldx=64, codes=P[1], ld_codes=32, scales=P[2], ld_scales=2, zeros=P[3],
             ld_zeros=2, bias=None, Y=P[4], ldy=8, workspace=P[5], workspace_bytes=1 << 24, stream=None)
    a.update(over)
    return dga.dga_q4_linear(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(dtype=gen.F32), 1), (dict(group=16), 1), (dict(group=0), 1), (dict(M=BIG), -2), (dict(N=-1), -3), (dict(K=-1), -4),
    (dict(X=None), -6), (dict(X=P[0] + 1), -6), (dict(ldx=63), -7), (dict(codes=None), -8), (dict(codes=P[1] + 8), -8),
    (dict(ld_codes=16), -9), (dict(ld_codes=40), -9), (dict(scales=None), -10), (dict(scales=P[2] + 1), -10), (dict(ld_scales=1), -11),
    (dict(ld_zeros=1), -13), (dict(bias=P[6] + 1), -14), (dict(Y=None), -15), (dict(ldy=7), -16), (dict(workspace=P[5] + 16), -17),
    (dict(Y=P[0]), 6), (dict(Y=P[1] + 64), 6), (dict(Y=P[2]), 6), (dict(Y=P[3]), 6), (dict(bias=P[4]), 6),
    (dict(M=0, X=None, Y=None), 0), (dict(N=0, codes=None, Y=None), 0)])
def test_q4_linear_arguments(over, code):
    assert _linear(**over) == code


def _q4_gated(**over):
    a = dict(dtype=gen.BF16, act=0, M=40, F=4, K=64, group=64, X=P[0], ldx=64, codes=P[1], ld_codes=32, scales=P[2], ld_scales=1, zeros=None,
             ld_zeros=0, bias=None, H=P[4], ldh=4, workspace=P[5], workspace_bytes=1 << 24, stream=None)
    a.update(over)
    return dga.dga_q4_gated(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(dtype=gen.F32), 1), (dict(act=7), 1), (dict(group=256), 1), (dict(M=-1), -3), (dict(F=BIG), -4), (dict(K=-1), -5), (dict(X=None), -7),
    (dict(ldx=63), -8), (dict(codes=None), -9), (dict(ld_codes=24), -10), (dict(scales=None), -11), (dict(ld_scales=0), -12),
    (dict(zeros=P[3], ld_zeros=0), -14), (dict(bias=P[6] + 1), -15), (dict(H=None), -16), (dict(ldh=3), -17), (dict(workspace=P[5] + 4), -18),
    (dict(H=P[1]), 6), (dict(F=0), 0)])
def test_q4_gated_arguments(over, code):
    assert _q4_gated(**over) == code


def _quantize(**over):
    a = dict(in_dtype=gen.F32, scale_dtype=gen.F16, rows=4, cols=40, group=32, W=P[0], ldw=40, codes=P[1], ld_codes=32, scales=P[2],
             ld_scales=2, zeros=P[3], ld_zeros=2, stream=None)
    a.update(over)
    return dga.dga_q4_quantize(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(in_dtype=gen.I8), 1), (dict(scale_dtype=gen.F32), 1), (dict(group=48), 1), (dict(rows=-1), -3), (dict(cols=BIG), -4), (dict(W=None), -6),
    (dict(ldw=39), -7), (dict(codes=P[1] + 1), -8), (dict(ld_codes=20), -9), (dict(scales=None), -10), (dict(ld_scales=1), -11),
    (dict(ld_zeros=1), -13), (dict(codes=P[0]), 6), (dict(scales=P[1]), 6), (dict(zeros=P[2]), 6), (dict(rows=0), 0)])
def test_q4_quantize_arguments(over, code):
    assert _quantize(**over) == code


@pytest.mark.parametrize("over,code", [
    (dict(scale_dtype=gen.F32), 1), (dict(out_dtype=gen.I8), 1), (dict(rows=-1), -3), (dict(cols=-1), -4), (dict(codes=None), -6), (dict(ld_codes=0), -7),
    (dict(scales=None), -8), (dict(ld_scales=1), -9), (dict(ld_zeros=0), -11), (dict(Y=None), -12), (dict(ldy=39), -13), (dict(Y=P[1]), 6)])
def test_q4_dequantize_arguments(over, code):
    a = dict(scale_dtype=gen.F16, out_dtype=gen.F32, rows=4, cols=40, group=32, codes=P[1], ld_codes=32, scales=P[2], ld_scales=2, zeros=P[3],
             ld_zeros=2, Y=P[4], ldy=40, stream=None)
    a.update(over)
    assert dga.dga_q4_dequantize(*a.values()) == code


def test_sizes_of_nothing_and_of_wrong_arguments():
    assert dga.dga_gated_workspace_size(gen.I8, 4, 4, 4, 4, 4, 0) == 0
    assert dga.dga_gated_workspace_size(gen.BF16, 0, 4, 4, 4, 4, 1) == 0
    assert dga.dga_gated_backward_workspace_size(gen.F16, 4, 0, 4, 4, 4) == 0
    assert dga.dga_q4_linear_workspace_size(gen.F32, 4, 4, 4, 4) == 0
    assert dga.dga_q4_gated_workspace_size(gen.F16, 4, -1, 4, 4) == 0
    # the gradient keeps dP: 16-bit values, rows of whole 16 bytes
    assert dga.dga_gated_backward_workspace_size(gen.F16, 100, 33, 64, 64, 64) >= 100 * 72 * 2


def test_a_short_workspace_is_refused():
    need = dga.dga_gated_backward_workspace_size(gen.F16, 40, 8, 16, 16, 16)
    assert need > 0 and _backward(workspace_bytes=need - 1) == dga.ERR_WORKSPACE
    need = dga.dga_gated_workspace_size(gen.F32, 40, 8, 16, 16, 16, 0)
    if need:
        assert _gated(dtype=gen.F32, M=40, workspace_bytes=need - 1) == dga.ERR_WORKSPACE


def test_python_refusals():
    X, W = torch.zeros(2, 4), torch.zeros(6, 4)
    with pytest.raises(ValueError):
        dga.gated_forward(X, W)  # not on a GPU
    with pytest.raises(ValueError):
        dga.gated_forward(X, W, activation="tanh")
    with pytest.raises(TypeError):
        dga.gated_forward(X.double(), W.double())
    with pytest.raises(ValueError):
        dga.gated_backward(X, W, torch.zeros(2, 6), torch.zeros(2, 3))
    with pytest.raises(TypeError):
        dga.q4_quantize(X.double())
    with pytest.raises(ValueError):
        dga.q4_quantize(X)
    codes, scales = torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        dga.q4_linear_forward(torch.zeros(1, 20, dtype=torch.float16), dga.Q4Tensor(20, 32, codes, scales))
    from dense_gemm_accelerator_gb300.q4 import _arguments
    for bad, error in ((dga.Q4Tensor(20, 48, codes, scales), ValueError), (dga.Q4Tensor(40, 32, codes, scales), ValueError),
                       (dga.Q4Tensor(20, 32, codes, scales.float()), TypeError), (dga.Q4Tensor(20, 32, codes.int(), scales), TypeError),
                       (dga.Q4Tensor(20, 32, codes, scales, scales), TypeError),
                       (dga.Q4Tensor(20, 32, codes, scales, torch.zeros(3, 2, dtype=torch.uint8)), ValueError),
                       (dga.Q4Tensor(20, 32, codes, scales.expand(3, 1).t().expand(3, 3)[:, :1].t(), None), ValueError),
                       (dga.Q4Tensor(20, 32, codes[:1].expand(3, 16), scales), ValueError)):
        with pytest.raises(error):
            _arguments(bad, codes.get_device())


# ---- the reference ------------------------------------------------------------------


def test_reference_activations_by_hand():
    x = torch.tensor([0.0, 1.0, -1.0, 3.0], dtype=torch.float64)
    phi = [0.5, 0.8413447460685429, 0.15865525393145707, 0.9986501019683699]
    s = [1 / (1 + math.exp(-v)) for v in x.tolist()]
    assert torch.allclose(ref.act(x, "gelu"), x * torch.tensor(phi, dtype=torch.float64), atol=1e-15)
    assert torch.allclose(ref.act(x, "silu"), x * torch.tensor(s, dtype=torch.float64), atol=1e-15)
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3))
    assert torch.allclose(ref.act(x, "gelu_tanh"), 0.5 * x * (1 + t), atol=1e-15)
    assert ref.act(x, "relu").tolist() == [0, 1, 0, 3] and ref.slope(x, "relu").tolist() == [0, 1, 0, 1]


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "sigmoid"])
def test_reference_slopes_are_differences(name):
    x = torch.linspace(-6, 6, 61, dtype=torch.float64)
    d = (ref.act(x + 1e-5, name) - ref.act(x - 1e-5, name)) / 2e-5
    assert torch.allclose(ref.slope(x, name), d, atol=1e-9)
    assert float(ref.slope(torch.linspace(-9, 9, 9001, dtype=torch.float64), name).abs().max()) < 1.13


def test_reference_quantisation_by_hand():
    w = torch.tensor([[-1.0, 0.0, 0.5, 2.0]])
    q, s, z = ref.q4_quantize(w, 32, True, torch.float16)  # s = 3/15 in fp16, z = 5
    assert s.item() == torch.tensor(0.2).half().item() and z.item() == 5
    assert q.tolist() == [[0, 5, 8, 15]]  # 0.5 / 0.19995 + 5 = 7.5006
    q, s, z = ref.q4_quantize(w, 32, False, torch.float16)
    assert s.item() == torch.tensor(2 / 7).half().item() and q.tolist() == [[4, 8, 10, 15]]  # -3.5004, 1.7502
    codes = torch.tensor([[0x50, 0xF8]], dtype=torch.uint8)
    assert ref.q4_unpack(codes, 4).tolist() == [[0, 5, 8, 15]]
    assert ref.q4_values(codes, torch.tensor([[0.5]]).half(), torch.tensor([[5]], dtype=torch.uint8), 3, 32).tolist() == [[-2.5, 0.0, 1.5]]


def test_layouts_of_the_cases():
    """The case file's packing is the format's."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operators", path)
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    w = torch.randn(5, 100, generator=torch.Generator().manual_seed(1))
    for zeros in (False, True):
        codes, s, z = cases._in_4_bits(w, 64, zeros, torch.float16)
        q, rs, rz = ref.q4_quantize(w, 64, zeros, torch.float16)
        assert torch.equal(ref.q4_unpack(codes, 100), q) and torch.equal(s, rs) and (z is None or torch.equal(z, rz))
