"""4-bit microscaled matrices: quantisation, products and the fully-connected
layer, as PyTorch-tensor forms of the ``dga_mx_*`` entry points (include/dga.h
has the formats, roundings and errors).  All work runs in the library's CUDA
kernels on the current stream of the tensors' device, or the one given;
scratch and results come from PyTorch's caching allocator, on the same stream.

NVFP4 needs a factor per tensor (``tensor_scale``, one float32 value on the
device; None is 1): under a factor f, blocks of magnitudes up to f / 170 become
zeros and magnitudes over 2688 f are held to 2688 f.  max|X| / 2688 takes the
whole range, and a power of two above it rounds nothing besides:

    r = (X.abs().amax().float() / 2688).reshape(1)
    f = torch.ldexp(torch.ones_like(r), torch.frexp(r).exponent)
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import BF16, F16, F32, DgaError, _check_lines, _elsewhere, _on_device, _raw_stream, lib, sum_rows

MXFP4, NVFP4 = 0, 1

_CODE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_TORCH = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}


# sizes of scratch and scales, by shape (a library call for one costs 0.7 us)
@functools.lru_cache(maxsize=4096)
def _scales_size(format, rows, K):
    return lib().dga_mx_scales_size(format, rows, K)


@functools.lru_cache(maxsize=4096)
def _linear_workspace(format, M, K):
    return lib().dga_mx_linear_workspace_size(format, M, K)


@functools.lru_cache(maxsize=4096)
def _backward_workspace(format, M, N, K):
    return lib().dga_mx_linear_backward_workspace_size(format, M, N, K)


class MXTensor:
    """A rows x cols matrix in 4 bits, quantised along its columns.

    codes: (rows, row_bytes) uint8, two E2M1 codes to a byte; scales: the tiled
    block scales; tensor_scale: a 1-element fp32 tensor, or None for 1."""
    __slots__ = ("format", "rows", "cols", "codes", "scales", "tensor_scale")

    def __init__(self, format, rows, cols, codes, scales, tensor_scale=None):
        self.format, self.rows, self.cols = format, rows, cols
        self.codes, self.scales, self.tensor_scale = codes, scales, tensor_scale

    @property
    def shape(self):
        return (self.rows, self.cols)

    @property
    def device(self):
        return self.codes.device

    def __repr__(self):
        return (f"MXTensor({'MXFP4' if self.format == MXFP4 else 'NVFP4'}, "
                f"{self.rows}x{self.cols}, {self.codes.device})")


def on_stream(stream, device, f, *args):
    """f(*args) with `stream` (an integer) as the current one, so that what it
    allocates belongs to that stream too: memory that the caller's stream still
    reads is not handed out again, and scratch is not freed under the work."""
    s = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(s):
        return f(*args)


def _raise(st, what):
    raise DgaError(st, what)


def _factor(t, format, device):
    """The device pointer of a tensor scale."""
    if t is None:
        return None
    if format != NVFP4:
        raise ValueError("tensor_scale needs the NVFP4 format")
    if t.dtype is not torch.float32 or t.numel() != 1 or t.device != device:
        raise ValueError("tensor_scale must be one float32 value on the tensor's device")
    return t.data_ptr()


def _rows_of(T, name):
    """(rows, columns, leading dimension) of a row-major 2-D tensor."""
    if T.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    (rows, cols), (ld, step) = T.shape, T.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major")
    if ld < cols:
        _check_lines(name, rows, cols, ld)
    return rows, cols, ld if ld > cols else (cols or 1)


def mx_quantize(X, format=MXFP4, transpose=False, tensor_scale=None, stream=None):
    """X (rows x cols, float32, bfloat16 or float16, row- or column-major) to an
    :class:`MXTensor` quantised along its rows, or, with transpose=True, the
    MXTensor of X's transpose (quantised along X's columns).  tensor_scale: X's
    factor (NVFP4)."""
    if stream is not None:
        return on_stream(stream, X.device, mx_quantize, X, format, transpose, tensor_scale)
    if _elsewhere(X.device):
        return _on_device(X.device, mx_quantize, X, format, transpose, tensor_scale)
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    code = _CODE.get(X.dtype)
    if code is None:
        raise TypeError("X must be float32, bfloat16 or float16")
    if not X.is_cuda:
        raise ValueError("X must be a CUDA tensor")
    if X.stride(1) != 1 and X.shape[1] > 1 and X.stride(0) == 1:
        X, transpose = X.t(), not transpose  # a column-major X is its transpose, row-major
    rows, cols, ldx = _rows_of(X, "X")
    R, K = (cols, rows) if transpose else (rows, cols)
    dev, L = X.device, lib()
    row_bytes = (K + 31) // 32 * 16  # dga_mx_row_bytes
    codes = torch.empty((R, row_bytes), dtype=torch.uint8, device=dev)
    scales = torch.empty(_scales_size(format, R, K), dtype=torch.uint8, device=dev)
    st = L.dga_mx_quantize(format, code, 1 if transpose else 0, rows, cols, X.data_ptr(), ldx,
                           _factor(tensor_scale, format, dev), codes.data_ptr(), row_bytes,
                           scales.data_ptr(), _raw_stream(dev.index))
    if st:
        _raise(st, "dga_mx_quantize")
    return MXTensor(format, R, K, codes, scales, tensor_scale)


def mx_dequantize(Q, out_dtype=F32, stream=None):
    """The values an MXTensor stands for, code * (scale * factor) in fp32, rounded
    to out_dtype."""
    if stream is not None:
        return on_stream(stream, Q.device, mx_dequantize, Q, out_dtype)
    dev = Q.codes.device
    if _elsewhere(dev):
        return _on_device(dev, mx_dequantize, Q, out_dtype)
    Y = torch.empty((Q.rows, Q.cols), dtype=_TORCH[out_dtype], device=dev)
    st = lib().dga_mx_dequantize(Q.format, out_dtype, Q.rows, Q.cols, Q.codes.data_ptr(),
                                 Q.codes.stride(0), Q.scales.data_ptr(),
                                 _factor(Q.tensor_scale, Q.format, dev), Y.data_ptr(), Q.cols or 1,
                                 _raw_stream(dev.index))
    if st:
        _raise(st, "dga_mx_dequantize")
    return Y


def _output(C, M, N, beta, out_dtype, device):
    """(the output, its type's code, its leading dimension)."""
    if C is None:
        if beta != 0:
            raise ValueError("beta != 0 needs C")
        return torch.empty((M, N), dtype=_TORCH[out_dtype], device=device), out_dtype, N or 1
    if tuple(C.shape) != (M, N) or C.dtype not in _CODE or C.device != device:
        raise ValueError(f"the output must be a ({M}, {N}) float32, bfloat16 or float16 tensor on {device}")
    return C, _CODE[C.dtype], _rows_of(C, "the output")[2]


def _bias(bias, N, C):
    if bias is None:
        return None
    if bias.dim() != 1 or bias.numel() != N or (N > 1 and bias.stride(0) != 1) or bias.dtype is not C.dtype \
            or bias.device != C.device:
        raise ValueError("bias must be a contiguous vector of the output's length, type and device")
    return bias.data_ptr()


def mx_gemm(A, B, C=None, alpha=1.0, beta=0.0, out_dtype=BF16, bias=None, stream=None):
    """C <- alpha * A @ B^T + beta * C (+ bias) of MXTensors A (M x K) and B
    (N x K) of one format; returns C, allocated as out_dtype when None."""
    if stream is not None:
        return on_stream(stream, A.device, mx_gemm, A, B, C, alpha, beta, out_dtype, bias)
    if A.format != B.format:
        raise TypeError("A and B must have the same format")
    if A.cols != B.cols:
        raise ValueError(f"shape mismatch: A {A.shape}, B {B.shape} (the products run along the columns)")
    if A.device != B.device:
        raise ValueError("A and B must be on the same device")
    dev = A.codes.device
    if _elsewhere(dev):
        return _on_device(dev, mx_gemm, A, B, C, alpha, beta, out_dtype, bias)
    C, code, ldc = _output(C, A.rows, B.rows, beta, out_dtype, dev)
    a, b = ctypes.c_float(alpha), ctypes.c_float(beta)
    st = lib().dga_mx_gemm(A.format, code, A.rows, B.rows, A.cols, ctypes.byref(a), A.codes.data_ptr(),
                           A.codes.stride(0), A.scales.data_ptr(), _factor(A.tensor_scale, A.format, dev),
                           B.codes.data_ptr(), B.codes.stride(0), B.scales.data_ptr(),
                           _factor(B.tensor_scale, B.format, dev), ctypes.byref(b), C.data_ptr(), ldc,
                           _bias(bias, B.rows, C), _raw_stream(dev.index))
    if st:
        _raise(st, "dga_mx_gemm")
    return C


def mx_linear_forward(X, W, bias=None, Y=None, tensor_scale=None, workspace=None, stream=None):
    """Y = X @ W^T + bias for X [batch, in] (float32, bfloat16 or float16) and a
    4-bit weight W, an MXTensor [out, in]: X is quantised in W's format
    (tensor_scale: its factor) and multiplied.  Y, of X's type unless given."""
    if stream is not None:
        return on_stream(stream, X.device, mx_linear_forward, X, W, bias, Y, tensor_scale, workspace)
    code = _CODE.get(X.dtype)
    if code is None:
        raise TypeError("X must be float32, bfloat16 or float16")
    shape = X.shape
    if len(shape) != 2 or shape[1] != W.cols:
        raise ValueError(f"shape mismatch: X {tuple(shape)}, W {W.shape}")
    M, K = shape
    ldx, step = X.stride()
    if step != 1 and K > 1:
        raise ValueError("X must be row-major")
    if ldx < K:
        _check_lines("X", M, K, ldx)
    dev, fmt, N, codes = X.device, W.format, W.rows, W.codes
    if codes.device != dev:
        raise ValueError("X and W must be on the same device")
    if _elsewhere(dev):
        return _on_device(dev, mx_linear_forward, X, W, bias, Y, tensor_scale, workspace)
    if Y is None:
        Y, out, ldy = torch.empty((M, N), dtype=X.dtype, device=dev), code, N or 1
    else:
        Y, out, ldy = _output(Y, M, N, 0, code, dev)
    L = lib()
    if workspace is None:
        have = _linear_workspace(fmt, M, K)  # 0 for a few rows
        if have:
            workspace = torch.empty(have, dtype=torch.uint8, device=dev)
    else:
        have = workspace.numel() * workspace.element_size()
    st = L.dga_mx_linear(fmt, code, out, M, N, K, X.data_ptr(), ldx if ldx > K else K or 1,
                         None if tensor_scale is None else _factor(tensor_scale, fmt, dev),
                         codes.data_ptr(), codes.stride(0), W.scales.data_ptr(),
                         None if W.tensor_scale is None else _factor(W.tensor_scale, fmt, dev),
                         None if bias is None else _bias(bias, N, Y), Y.data_ptr(), ldy,
                         workspace.data_ptr() if have else None, have, _raw_stream(dev.index))
    if st:
        _raise(st, "dga_mx_linear")
    return Y


def mx_linear_backward(X, W, G, format=MXFP4, tensor_scales=(None, None, None), need_bias=True, stream=None):
    """Gradients of Y = X W^T + b for the output gradient G [batch, out], with
    4-bit products (the roundings' own gradient taken as 1): dX = G W with G
    and W quantised along out, dW = G^T X with G and X quantised along the
    batch, both of G's type; db = the batch sum of G (fp32, unquantised).
    tensor_scales: the factors of X, W and G (NVFP4: without them gradients
    near 1e-3 and below are quantised to zeros)."""
    if stream is not None:
        return on_stream(stream, G.device, mx_linear_backward, X, W, G, format, tensor_scales, need_bias)
    if X.shape[0] != G.shape[0] or X.shape[1] != W.shape[1] or G.shape[1] != W.shape[0]:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, G {tuple(G.shape)}")
    if G.dtype not in _CODE:
        raise TypeError("G must be float32, bfloat16 or float16")
    sx, sw, sg = tensor_scales
    out, dev = _CODE[G.dtype], G.device
    if _elsewhere(dev):
        return _on_device(dev, mx_linear_backward, X, W, G, format, tensor_scales, need_bias)
    if all(T.stride(1) == 1 and T.is_cuda and T.device == dev and T.dtype in _CODE for T in (X, W, G)):
        (M, N, ldg), (_, K, ldx), (_, _, ldw) = _rows_of(G, "G"), _rows_of(X, "X"), _rows_of(W, "W")
        dX = torch.empty((M, K), dtype=G.dtype, device=dev)
        dW = torch.empty((N, K), dtype=G.dtype, device=dev)
        db = torch.empty(N, dtype=torch.float32, device=dev) if need_bias else None
        L = lib()
        have = _backward_workspace(format, M, N, K)
        workspace = torch.empty(have, dtype=torch.uint8, device=dev) if have else None
        st = L.dga_mx_linear_backward(format, _CODE[X.dtype], _CODE[W.dtype], out, M, N, K, X.data_ptr(),
                                      ldx, _factor(sx, format, dev), W.data_ptr(),
                                      ldw, _factor(sw, format, dev), G.data_ptr(),
                                      ldg, _factor(sg, format, dev), dX.data_ptr(), K or 1,
                                      dW.data_ptr(), K or 1, db.data_ptr() if need_bias else None,
                                      workspace.data_ptr() if have else None, have, _raw_stream(dev.index))
        if st:
            _raise(st, "dga_mx_linear_backward")
        return dX, dW, db
    # column-major operands, which are quantised along the other axis
    dX = mx_gemm(mx_quantize(G, format, False, sg), mx_quantize(W, format, True, sw), out_dtype=out)
    dW = mx_gemm(mx_quantize(G, format, True, sg), mx_quantize(X, format, True, sx), out_dtype=out)
    if not need_bias:
        return dX, dW, None
    return dX, dW, sum_rows(G if G.stride(1) == 1 or G.shape[1] <= 1 else G.contiguous())  # along its rows
