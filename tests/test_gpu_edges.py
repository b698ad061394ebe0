"""Edges of the 4-bit and orthogonalisation calls on the GPU: zero tensors,
values far past a tensor's factor, host threads, devices and eps = 0."""

import numpy as np
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

FMT = [dga.MXFP4, dga.NVFP4]
TYPES = [torch.float32, torch.bfloat16, torch.float16]
OUT = {torch.float32: dga.F32, torch.bfloat16: dga.BF16, torch.float16: dga.F16}


def _parts(q):
    """(codes, scale bytes) of an MXTensor on the host."""
    return (ref.unpack_codes(q.codes.cpu().numpy(), q.cols),
            ref.untile_scales(q.scales.cpu().numpy(), q.rows, q.cols, q.format))


def _sync_ok():
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 13, 40, 300])
def test_a_zero_tensor_with_its_zero_factor(dtype, rows):
    """max|X| / 2688 of a zero tensor is 0: its blocks are zeros still."""
    N, K = 130, 200
    zero = torch.zeros(1, device="cuda")
    X = torch.zeros(rows, K, dtype=dtype, device="cuda")
    X[0, 3] = -0.0
    for transpose in (False, True):
        q = dga.mx_quantize(X, dga.NVFP4, transpose=transpose, tensor_scale=zero)
        codes, scales = _parts(q)
        assert not scales.any() and not (codes & 7).any()
        assert not dga.mx_dequantize(q).any()
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(1)).cuda()
    W = dga.mx_quantize(w, dga.NVFP4)
    bias = torch.arange(N, device="cuda").to(dtype)
    assert torch.equal(dga.mx_linear_forward(X, W, bias, tensor_scale=zero), bias.expand(rows, N))
    G = torch.randn(rows, N, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    dX, dW, db = dga.mx_linear_backward(X, w, G, dga.NVFP4, tensor_scales=(zero, None, None))
    assert not dW.any() and bool(torch.isfinite(dX).all())
    dX, dW, db = dga.mx_linear_backward(X, w, torch.zeros_like(G), dga.NVFP4, tensor_scales=(zero, None, zero))
    _sync_ok()
    assert not dX.any() and not dW.any() and not db.any()


def test_zero_blocks_beside_others_keep_a_zero_scale():
    X = torch.zeros(4, 64, device="cuda")
    X[1, 16:32] = 3.0
    for f in (None, torch.full((1,), 2.0 ** -120, device="cuda"), torch.full((1,), 2.0 ** 120, device="cuda")):
        _, scales = _parts(dga.mx_quantize(X, dga.NVFP4, tensor_scale=f))
        want = np.zeros((4, 4), np.uint8)
        want[1, 1] = ref.quantize(X.cpu().double().numpy(), dga.NVFP4, 1.0 if f is None else float(f))[1][1, 1]
        assert np.array_equal(scales, want)
