"""4-bit weights with group scales, and products with 16-bit activations:
PyTorch-tensor forms of the ``dga_q4_*`` entry points (include/dga.h has the
format, roundings and errors).  Unlike the microscaled matrices of ``mx``, only
the weight is held in 4 bits: activations are multiplied as they are.  All work
runs in the library's CUDA kernels on the current stream of the tensors' device,
or the one given; scratch and results come from PyTorch's caching allocator, on
the same stream.
"""
from __future__ import annotations

import functools

import torch

from . import F32, DgaError, _check_lines, _current_device, _elsewhere, _on_device, _raw_stream, lib
from .gated import activation_code, result, scratch, vector
from .mx import _CODE, _TORCH, _rows_of, on_stream

_U8 = torch.uint8
_HALF = {torch.bfloat16: _CODE[torch.bfloat16], torch.float16: _CODE[torch.float16]}


# sizes of scratch, by shape and by the (current) device
@functools.lru_cache(maxsize=4096)
def _linear_workspace(device, code, M, N, K, ldx):
    return lib().dga_q4_linear_workspace_size(code, M, N, K, ldx)


@functools.lru_cache(maxsize=4096)
def _gated_workspace(device, code, M, F, K, ldx):
    return lib().dga_q4_gated_workspace_size(code, M, F, K, ldx)


class Q4Tensor:
    """A weight of `cols` columns in 4 bits, w = (q - z) * s per row and group of 32,
    64 or 128 columns: codes (rows, at least ceil(cols / 32) * 16) uint8, column k in byte
    k // 2, the even one in the low half; scales (rows, ceil(cols / group)) bfloat16 or
    float16; zeros of the same shape, uint8, or None for 8 throughout."""
    __slots__ = ("cols", "group", "codes", "scales", "zeros")

    def __init__(self, cols, group, codes, scales, zeros=None):
        self.cols, self.group = cols, group
        self.codes, self.scales, self.zeros = codes, scales, zeros

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def shape(self):
        return (self.codes.shape[0], self.cols)

    @property
    def device(self):
        return self.codes.device

    def __repr__(self):
        return f"Q4Tensor({self.rows}x{self.cols}, groups of {self.group}, {self.codes.device})"


def _arguments(Q, d):
    """(rows, code of the scales' type, the weight's arguments of the C calls); d: the
    number of the device that it must be on.  (The checks cost a call 2 us.)"""
    codes, scales, zeros, cols, group = Q.codes, Q.scales, Q.zeros, Q.cols, Q.group
    code = _HALF.get(scales.dtype)
    if code is None:
        raise TypeError("scales must be bfloat16 or float16")
    if codes.dtype is not _U8:
        raise TypeError("codes must be uint8")
    if group != 128 and group != 64 and group != 32:
        raise ValueError("groups have 32, 64 or 128 columns")
    (rows, width), (lc, one) = codes.shape, codes.stride()
    shape, (ls, step) = scales.shape, scales.stride()
    groups = (cols + group - 1) // group
    if shape[0] != rows or shape[1] != groups or width < (cols + 31) // 32 * 16:
        raise ValueError(f"a {rows} x {cols} weight in groups of {group} has codes ({rows}, {(cols + 31) // 32 * 16}) and "
                         f"scales ({rows}, {groups}), not {tuple(codes.shape)} and {tuple(shape)}")
    if codes.get_device() != d or scales.get_device() != d:
        raise ValueError("the weight's tensors must be on the device of X")
    if (one != 1 and width > 1) or (step != 1 and groups > 1):
        raise ValueError("codes and scales must be row-major")
    if lc < width:
        _check_lines("codes", rows, width, lc)
        lc = width
    if ls < groups:
        _check_lines("scales", rows, groups, ls)
        ls = groups
    if zeros is None:
        return rows, code, codes.data_ptr(), lc, scales.data_ptr(), ls, None, 0
    if zeros.dtype is not _U8:
        raise TypeError("zeros must be uint8")
    if zeros.shape != shape or zeros.get_device() != d:
        raise ValueError("zeros must have the shape and device of the scales")
    lz, step = zeros.stride()
    if step != 1 and groups > 1:
        raise ValueError("zeros must be row-major")
    if lz < groups:
        _check_lines("zeros", rows, groups, lz)
        lz = groups
    return rows, code, codes.data_ptr(), lc, scales.data_ptr(), ls, zeros.data_ptr(), lz


def q4_quantize(W, group=128, zeros=True, scale_dtype=None, stream=None):
    """W (rows x cols, float32, bfloat16 or float16, row-major) to a :class:`Q4Tensor`
    with a zero point per group (zeros=True), or symmetric about 8; scales of
    scale_dtype, W's own 16-bit type or bfloat16 unless given."""
    if stream is not None:
        return on_stream(stream, W.device, q4_quantize, W, group, zeros, scale_dtype)
    code = _CODE.get(W.dtype)
    if code is None:
        raise TypeError("W must be float32, bfloat16 or float16")
    if not W.is_cuda:
        raise ValueError("W must be a CUDA tensor")
    if group not in (32, 64, 128):
        raise ValueError("groups have 32, 64 or 128 columns")
    if scale_dtype is None:
        scale_dtype = W.dtype if W.dtype in _HALF else torch.bfloat16
    if scale_dtype not in _HALF:
        raise TypeError("scale_dtype must be bfloat16 or float16")
    dev = W.device
    if _elsewhere(dev):
        return _on_device(dev, q4_quantize, W, group, zeros, scale_dtype)
    rows, cols, ldw = _rows_of(W, "W")
    width, groups = (cols + 31) // 32 * 16, -(-cols // group)
    codes = torch.empty((rows, width), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, groups), dtype=scale_dtype, device=dev)
    z = torch.empty((rows, groups), dtype=torch.uint8, device=dev) if zeros else None
    st = lib().dga_q4_quantize(code, _HALF[scale_dtype], rows, cols, group, W.data_ptr(), ldw, codes.data_ptr(), width,
                               scales.data_ptr(), groups, z.data_ptr() if zeros else None, groups, _raw_stream(dev.index))
    if st:
        raise DgaError(st, "dga_q4_quantize")
    return Q4Tensor(cols, group, codes, scales, z)


def q4_dequantize(Q, out_dtype=F32, stream=None):
    """The values a Q4Tensor stands for, (q - z) * s, rounded to out_dtype: among others
    what gradients through a frozen 4-bit weight multiply by."""
    if stream is not None:
        return on_stream(stream, Q.device, q4_dequantize, Q, out_dtype)
    dev = Q.codes.device
    if dev.type != "cuda":
        raise ValueError("Q must be on a CUDA device")
    if _elsewhere(dev):
        return _on_device(dev, q4_dequantize, Q, out_dtype)
    rows, code, c, lc, s, ls, z, lz = _arguments(Q, dev.index)
    Y = torch.empty((rows, Q.cols), dtype=_TORCH[out_dtype], device=dev)
    st = lib().dga_q4_dequantize(code, out_dtype, rows, Q.cols, Q.group, c, lc, s, ls, z, lz, Y.data_ptr(), Q.cols or 1,
                                 _raw_stream(dev.index))
    if st:
        raise DgaError(st, "dga_q4_dequantize")
    return Y


def _rows_for(X, Q):
    """(M, K, ldx) of activations for a weight."""
    if X.dtype is not Q.scales.dtype:
        raise TypeError("X must have the type of the weight's scales (bfloat16 or float16)")
    shape = X.shape
    if len(shape) != 2 or shape[1] != Q.cols:
        raise ValueError(f"shape mismatch: X {tuple(shape)}, the weight {Q.shape}")
    M, K = shape
    ldx, step = X.stride()
    if step != 1 and K > 1:
        raise ValueError("X must be row-major")
    if ldx < K:
        _check_lines("X", M, K, ldx)
    return M, K, ldx if ldx > K else K or 1


def q4_linear_forward(X, W, bias=None, Y=None, workspace=None, stream=None):
    """Y = X @ W^T + bias for X [batch, in] and a 4-bit weight W, a Q4Tensor [out, in];
    X, the scales, the bias and Y of one type, bfloat16 or float16.  Up to 32 rows
    (64 of smaller weights) multiply the codes as they are; more go through W's values
    rounded to X's type."""
    if stream is not None:
        return on_stream(stream, X.device, q4_linear_forward, X, W, bias, Y, workspace)
    d = X.get_device()
    if d < 0:
        raise ValueError("X must be a CUDA tensor")
    if d != _current_device():
        return _on_device(X.device, q4_linear_forward, X, W, bias, Y, workspace)
    M, K, ldx = _rows_for(X, W)
    N, code, c, lc, s, ls, z, lz = _arguments(W, d)
    if Y is None:
        Y, ldy = torch.empty((M, N), dtype=X.dtype, device=d), N or 1
    else:
        Y, ldy = result(Y, M, N, X.dtype, X.device, "Y")
    x = X.data_ptr()
    if workspace is None:
        have = _linear_workspace(d, code, M, N, K, ldx if x % 16 == 0 else ldx | 1) if M > 512 or ldx % 8 or x % 16 or not K else 0
        if have:
            workspace = torch.empty(have, dtype=_U8, device=d)
    else:
        have = scratch(workspace, d)
    st = lib().dga_q4_linear(code, M, N, K, W.group, x, ldx, c, lc, s, ls, z, lz,
                             None if bias is None else vector(bias, N, X.dtype, X.device), Y.data_ptr(), ldy,
                             workspace.data_ptr() if have else None, have, _raw_stream(d))
    if st:
        raise DgaError(st, "dga_q4_linear")
    return Y


def q4_gated_forward(X, W, bias=None, activation="silu", H=None, workspace=None, stream=None):
    """The gated layer H = act(g) * u, [g | u] = X @ W^T + bias, on a 4-bit weight W, a
    Q4Tensor [2 * hidden, in] (the gate's rows first); types as for q4_linear_forward,
    activations as for gated_forward."""
    if stream is not None:
        return on_stream(stream, X.device, q4_gated_forward, X, W, bias, activation, H, workspace)
    d, act = X.get_device(), activation_code(activation)
    if d < 0:
        raise ValueError("X must be a CUDA tensor")
    if d != _current_device():
        return _on_device(X.device, q4_gated_forward, X, W, bias, activation, H, workspace)
    M, K, ldx = _rows_for(X, W)
    N, code, c, lc, s, ls, z, lz = _arguments(W, d)
    if N % 2:
        raise ValueError("the weight must have an even number of rows")
    F = N // 2
    if H is None:
        H, ldh = torch.empty((M, F), dtype=X.dtype, device=d), F or 1
    else:
        H, ldh = result(H, M, F, X.dtype, X.device, "H")
    x = X.data_ptr()
    if workspace is None:
        have = _gated_workspace(d, code, M, F, K, ldx if x % 16 == 0 else ldx | 1) if M > 512 or ldx % 8 or x % 16 or not K else 0
        if have:
            workspace = torch.empty(have, dtype=_U8, device=d)
    else:
        have = scratch(workspace, d)
    st = lib().dga_q4_gated(code, act, M, F, K, W.group, x, ldx, c, lc, s, ls, z, lz,
                            None if bias is None else vector(bias, N, X.dtype, X.device), H.data_ptr(), ldh,
                            workspace.data_ptr() if have else None, have, _raw_stream(d))
    if st:
        raise DgaError(st, "dga_q4_gated")
    return H
