"""Orthogonalised updates (the Muon optimiser's step) as a PyTorch-tensor form of
``dga_orthogonalize`` (include/dga.h has the iteration, numerics and errors)."""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F16, F32, DgaError, _check_lines, _elsewhere, _on_device, _raw_stream, lib
from .mx import on_stream

_CODE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_TORCH = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}

#: a, b, c of X <- a X + (b A + c A^2) X: K. Jordan, "Muon: An optimizer for
#: hidden layers in neural networks" (2024)
QUINTIC = (3.4445, -4.7750, 2.0315)


def _layout(T, name):
    """(batch, rows, columns, leading dimension, matrix stride) of a 2-D or 3-D
    tensor whose rows are contiguous."""
    shape, stride = T.shape, T.stride()
    rows, cols = shape[-2], shape[-1]
    if stride[-1] != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    _check_lines(name, rows, cols, stride[-2])
    ld = stride[-2] if rows > 1 else cols
    return (1, rows, cols, ld, 0) if len(shape) == 2 else (shape[0], rows, cols, ld, stride[0])


def orthogonalize(G, steps=5, coefficients=QUINTIC, eps=1e-7, out=None, out_dtype=None,
                  workspace=None, stream=None):
    """G (rows x cols, or a batch of such matrices) orthogonalised by `steps`
    Newton-Schulz steps: every singular value towards 1.

    bfloat16 results of more than 256 rows and columns come from products of
    11-bit operands (up to 1.7e-3 off, as much as their own rounding); float32
    ones, with out_dtype=F32, from 22-bit operands.

    coefficients: (a, b, c) for all steps, or one such triple per step.  out:
    the result, of G's shape (it may be G itself), allocated as out_dtype (G's
    own type if None) when None.  The workspace comes from PyTorch's caching
    allocator unless given (dga_orthogonalize_workspace_size bytes)."""
    if stream is not None:
        return on_stream(stream, G.device, orthogonalize, G, steps, coefficients, eps, out, out_dtype, workspace)
    if G.dim() not in (2, 3):
        raise ValueError("G must be a matrix or a batch of matrices")
    code = _CODE.get(G.dtype)
    if code is None:
        raise TypeError("G must be float32, bfloat16 or float16")
    if not G.is_cuda:
        raise ValueError("G must be a CUDA tensor")
    dev = G.device
    if _elsewhere(dev):
        return _on_device(dev, orthogonalize, G, steps, coefficients, eps, out, out_dtype, workspace)
    if out is None:
        out_code = code if out_dtype is None else out_dtype
        out = torch.empty(G.shape, dtype=_TORCH[out_code], device=dev)
    elif out.shape != G.shape or out.dtype not in _CODE or out.device != dev:
        raise ValueError("out must be a float32, bfloat16 or float16 tensor of G's shape, on its device")
    else:
        out_code = _CODE[out.dtype]
    if hasattr(coefficients[0], "__len__"):
        flat = [c for t in coefficients for c in t]
    else:
        flat = list(coefficients) * max(steps, 0)
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients must be one (a, b, c), or {steps} of them")
    batch, rows, cols, ldg, stride_g = _layout(G, "G")
    _, _, _, ldo, stride_o = _layout(out, "out")
    L = lib()
    need = L.dga_orthogonalize_workspace_size(out_code, batch, rows, cols)
    if workspace is None:
        workspace, have = torch.empty(need, dtype=torch.uint8, device=dev), need
    else:
        have = workspace.numel() * workspace.element_size()
    st = L.dga_orthogonalize(code, out_code, batch, rows, cols, G.data_ptr(), ldg, stride_g, out.data_ptr(),
                             ldo, stride_o, steps, (ctypes.c_float * len(flat))(*flat), eps,
                             workspace.data_ptr() or None, have,
                             _raw_stream(dev.index))
    if st:
        raise DgaError(st, "dga_orthogonalize")
    return out
