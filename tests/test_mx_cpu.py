"""The 4-bit and orthogonalisation entry points without a GPU: sizes, argument
errors (reported before the device is touched), and the test reference of the
formats against hand-written cases."""
import ctypes

import numpy as np
import pytest

import dense_gemm_accelerator_gb300 as dga
from dense_gemm_accelerator_gb300 import build as dga_build
from dense_gemm_accelerator_gb300 import inputs as gen
from tests import mx_reference as ref

A, B, C, D, E = (0x10000000 * i for i in range(1, 6))  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    dga_build.build()
    return dga.lib()


# ---- the reference ------------------------------------------------------------------


def test_e2m1_ties_go_to_the_even_code():
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 0.2500001, 7.9, 0.0]])
    codes, scales = ref.quantize(x, ref.MX)
    assert scales[0, 0] == 127  # 2^0: floor(log2 7.9) - 2
    assert codes[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 1, 7, 0]


def test_mx_scales_by_hand():
    for m, byte in ((1.0, 125), (6.0, 127), (7.999, 127), (8.0, 128), (2.0 ** -126, 0), (0.0, 0), (3.4e38, 252), (np.inf, 255), (np.nan, 255)):
        assert ref.quantize(np.array([[m]]), ref.MX)[1][0, 0] == byte, m


def test_nv_scales_by_hand():
    assert ref.E4M3[-1] == 448.0 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6
    for m, byte in ((6.0, 56), (6.0 * 448, 126), (1e9, 126), (0.0, 0), (6 * 1.0625, 56), (6 * 1.1875, 58), (np.nan, 127)):
        assert ref.quantize(np.array([[m]]), ref.NV)[1][0, 0] == byte, m  # 1.0625 and 1.1875 are ties


def test_scale_tiles_are_a_permutation():
    for fmt in (ref.MX, ref.NV):
        rows, K = 300, 1000
        n = -(-K // ref.BLOCK[fmt])
        size = dga.dga_mx_scales_size(fmt, rows, K)
        got = ref.untile_scales(np.arange(size), rows, K, fmt)
        assert size == 384 * -(-n // 4) * 4 and len(np.unique(got)) == rows * n


# ---- sizes -----------------------------------------------------------------------------


@pytest.mark.parametrize("K,row", [(0, 0), (1, 16), (32, 16), (33, 32), (1000, 512), (4096, 2048)])
def test_row_bytes(K, row):
    assert dga.dga_mx_row_bytes(K) == row


def test_workspace_sizes():
    assert dga.dga_mx_linear_workspace_size(dga.MXFP4, 16, 4096) == 0  # the product quantises
    assert dga.dga_mx_linear_workspace_size(dga.MXFP4, 17, 4096) == 17 * 2048 + 128 * 128
    assert dga.dga_mx_linear_workspace_size(dga.NVFP4, 300, 100) == 300 * 64 + 3 * 2 * 512
    assert dga.dga_mx_scales_size(dga.MXFP4, 0, 5) == 0 and dga.dga_mx_scales_size(7, 5, 5) == 0
    small = dga.dga_orthogonalize_workspace_size(gen.BF16, 1, 1024, 1024)
    assert 0 < small < dga.dga_orthogonalize_workspace_size(gen.F32, 1, 1024, 1024)  # lo words of A and B
    assert dga.dga_orthogonalize_workspace_size(gen.F32, 0, 4, 4) == 0
    assert dga.dga_orthogonalize_workspace_size(gen.F32, 1, 4, 9) == dga.dga_orthogonalize_workspace_size(gen.F32, 1, 9, 4)


# ---- refusals ----------------------------------------------------------------------------


def _quantize(**over):
    a = dict(format=dga.NVFP4, in_dtype=gen.BF16, transpose=0, rows=4, cols=64, X=A, ldx=64, tensor_scale=None,
             codes=B, ld_codes=32, scales=C, stream=None)
    a.update(over)
    return dga.dga_mx_quantize(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(format=2), dga.ERR_UNSUPPORTED), (dict(in_dtype=gen.I8), dga.ERR_UNSUPPORTED), (dict(transpose=2), -3),
    (dict(rows=-1), -4), (dict(rows=1 << 30), -4), (dict(cols=-1), -5), (dict(X=None), -6), (dict(ldx=63), -7),
    (dict(format=dga.MXFP4, tensor_scale=D), -8), (dict(codes=None), -9), (dict(codes=B + 8), -9),
    (dict(ld_codes=16), -10), (dict(ld_codes=40), -10), (dict(transpose=1, ld_codes=8), -10), (dict(scales=None), -11),
    (dict(scales=C + 4), -11), (dict(codes=A), dga.ERR_OVERLAP), (dict(scales=A), dga.ERR_OVERLAP),
    (dict(scales=B), dga.ERR_OVERLAP), (dict(rows=0, X=None, codes=None), dga.OK), (dict(cols=0), dga.OK),
])
def test_quantize_arguments(over, code):
    assert _quantize(**over) == code


def _dequantize(**over):
    a = dict(format=dga.MXFP4, out_dtype=gen.F32, rows=4, cols=64, codes=B, ld_codes=32, scales=C, tensor_scale=None,
             Y=A, ldy=64, stream=None)
    a.update(over)
    return dga.dga_mx_dequantize(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(format=-1), dga.ERR_UNSUPPORTED), (dict(out_dtype=gen.I32), dga.ERR_UNSUPPORTED), (dict(rows=-1), -3),
    (dict(cols=-2), -4), (dict(codes=None), -5), (dict(ld_codes=31), -6), (dict(scales=C + 1), -7),
    (dict(tensor_scale=D), -8), (dict(Y=None), -9), (dict(ldy=63), -10), (dict(Y=B), dga.ERR_OVERLAP),
    (dict(cols=0, Y=None), dga.OK),
])
def test_dequantize_arguments(over, code):
    assert _dequantize(**over) == code


def _gemm(**over):
    one, zero = ctypes.c_float(1.0), ctypes.c_float(0.0)
    a = dict(format=dga.NVFP4, out_dtype=gen.BF16, M=4, N=5, K=64, alpha=ctypes.byref(one), A=A, lda=32, As=A + 4096,
             At=None, B=B, ldb=32, Bs=B + 4096, Bt=None, beta=ctypes.byref(zero), C=C, ldc=5, bias=None, stream=None)
    a.update(over)
    return dga.dga_mx_gemm(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(format=3), dga.ERR_UNSUPPORTED), (dict(out_dtype=gen.I8), dga.ERR_UNSUPPORTED), (dict(M=-1), -3), (dict(N=-1), -4),
    (dict(K=-1), -5), (dict(alpha=None), -6), (dict(A=None), -7), (dict(lda=31), -8), (dict(As=None), -9),
    (dict(format=dga.MXFP4, At=D), -10), (dict(B=B + 1), -11), (dict(ldb=0), -12), (dict(Bs=B + 4100), -13),
    (dict(format=dga.MXFP4, Bt=D), -14), (dict(beta=None), -15), (dict(C=None), -16), (dict(ldc=4), -17),
    (dict(C=A), dga.ERR_OVERLAP), (dict(C=B + 4096), dga.ERR_OVERLAP), (dict(bias=C), dga.ERR_OVERLAP),
    (dict(M=0, A=None), dga.OK), (dict(N=0, C=None), dga.OK),
])
def test_gemm_arguments(over, code):
    assert _gemm(**over) == code


def _linear(**over):
    a = dict(format=dga.NVFP4, x_dtype=gen.BF16, out_dtype=gen.BF16, M=20, N=5, K=64, X=A, ldx=64, xt=None, W=B, ldw=32,
             Ws=B + 4096, Wt=None, bias=None, Y=C, ldy=5, ws=D, ws_bytes=1 << 20, stream=None)
    a.update(over)
    return dga.dga_mx_linear(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(x_dtype=gen.I8), dga.ERR_UNSUPPORTED), (dict(M=-1), -4), (dict(N=-1), -5), (dict(K=-1), -6), (dict(X=None), -7),
    (dict(ldx=63), -8), (dict(format=dga.MXFP4, xt=E), -9), (dict(W=None), -10), (dict(ldw=16), -11), (dict(Ws=None), -12),
    (dict(format=dga.MXFP4, Wt=E), -13), (dict(Y=None), -15), (dict(ldy=4), -16), (dict(ws=None), -17), (dict(ws=D + 8), -17),
    (dict(ws_bytes=100), dga.ERR_WORKSPACE), (dict(ws=None, ws_bytes=0), dga.ERR_WORKSPACE), (dict(Y=A), dga.ERR_OVERLAP),
    (dict(ws=A), dga.ERR_OVERLAP), (dict(ws=B), dga.ERR_OVERLAP), (dict(Y=D), dga.ERR_OVERLAP), (dict(M=0), dga.OK),
])
def test_linear_arguments(over, code):
    assert _linear(**over) == code


def _backward(**over):
    a = dict(format=dga.NVFP4, x_dtype=gen.BF16, w_dtype=gen.F32, g_dtype=gen.F16, M=20, N=5, K=64, X=A, ldx=64, xt=None,
             W=B, ldw=64, wt=None, G=C, ldg=5, gt=None, dX=D, lddx=64, dW=E, lddw=64, db=E + (1 << 20), ws=E + (1 << 24),
             ws_bytes=1 << 20, stream=None)
    a.update(over)
    return dga.dga_mx_linear_backward(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(format=7), dga.ERR_UNSUPPORTED), (dict(w_dtype=gen.I8), dga.ERR_UNSUPPORTED), (dict(M=-1), -5), (dict(N=-1), -6),
    (dict(K=1 << 30), -7), (dict(X=None), -8), (dict(ldx=63), -9), (dict(format=dga.MXFP4, xt=A), -10), (dict(W=None), -11),
    (dict(ldw=63), -12), (dict(format=dga.MXFP4, wt=A), -13), (dict(G=None), -14), (dict(ldg=4), -15),
    (dict(format=dga.MXFP4, gt=A), -16), (dict(dX=None), -17), (dict(lddx=63), -18), (dict(dW=None), -19), (dict(lddw=63), -20),
    (dict(ws=None), -22), (dict(ws=E + (1 << 24) + 16), -22), (dict(ws_bytes=1000), dga.ERR_WORKSPACE),
    (dict(ws=None, ws_bytes=0), dga.ERR_WORKSPACE), (dict(dX=A), dga.ERR_OVERLAP), (dict(dX=C), dga.ERR_OVERLAP),
    (dict(dW=B + 256), dga.ERR_OVERLAP), (dict(dW=D), dga.ERR_OVERLAP), (dict(db=C), dga.ERR_OVERLAP), (dict(db=D), dga.ERR_OVERLAP),
    (dict(ws=A), dga.ERR_OVERLAP), (dict(ws=D), dga.ERR_OVERLAP),
])
def test_linear_backward_arguments(over, code):
    assert _backward(**over) == code


def test_linear_backward_workspace():
    size = dga.dga_mx_linear_backward_workspace_size
    assert size(dga.MXFP4, 0, 5, 7) == size(dga.NVFP4, 5, 0, 7) == size(dga.MXFP4, 5, 7, -1) == size(9, 1, 1, 1) == 0
    # G and W^T along 64, G^T and X^T along 32: codes in multiples of 256 bytes, scale tiles of 512
    assert size(dga.MXFP4, 32, 64, 48) == (32 * 32 + 512) + (48 * 32 + 512) + (64 * 16 + 512) + (48 * 16 + 512)


def _ortho(**over):
    a = dict(in_dtype=gen.F32, out_dtype=gen.F32, batch=2, rows=4, cols=8, G=A, ldg=8, stride_g=32, O=B, ldo=8, stride_o=32,
             steps=5, co=(ctypes.c_float * 15)(), eps=1e-7, ws=D, ws_bytes=1 << 24, stream=None)
    a.update(over)
    return dga.dga_orthogonalize(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(in_dtype=gen.I8), dga.ERR_UNSUPPORTED), (dict(out_dtype=gen.TF32), dga.ERR_UNSUPPORTED), (dict(batch=-1), -3),
    (dict(batch=65536), -3), (dict(rows=-1), -4), (dict(cols=-1), -5), (dict(G=None), -6), (dict(ldg=7), -7),
    (dict(stride_g=-1), -8), (dict(O=None), -9), (dict(ldo=7), -10), (dict(stride_o=31), -11), (dict(steps=0), -12),
    (dict(steps=1001), -12), (dict(co=None), -13), (dict(eps=-1.0), -14), (dict(eps=float("nan")), -14), (dict(ws=None), -15),
    (dict(ws=D + 16), -15), (dict(ws_bytes=256), dga.ERR_WORKSPACE), (dict(ws=A), dga.ERR_OVERLAP), (dict(ws=B), dga.ERR_OVERLAP),
    (dict(O=A + 16), dga.ERR_OVERLAP), (dict(O=A, out_dtype=gen.BF16), dga.ERR_OVERLAP), (dict(batch=0), dga.OK),
    (dict(rows=0, G=None), dga.OK),
])
def test_orthogonalize_arguments(over, code):
    assert _ortho(**over) == code
