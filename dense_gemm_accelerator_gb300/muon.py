"""Orthogonalised updates (the Muon optimiser's step) as a PyTorch-tensor form of
``dga_orthogonalize`` (include/dga.h has the iteration, numerics and errors)."""
from __future__ import annotations

import ctypes

import torch

from . import BF16, F16, F32, OK, DgaError, dga_orthogonalize_workspace_size, lib

_CODE = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_TORCH = {F32: torch.float32, BF16: torch.bfloat16, F16: torch.float16}

#: a, b, c of X <- a X + (b A + c A^2) X: K. Jordan, "Muon: An optimizer for
#: hidden layers in neural networks" (2024)
QUINTIC = (3.4445, -4.7750, 2.0315)


def _layout(T, name):
    """(batch, leading dimension, matrix stride) of a 2-D or 3-D tensor whose rows are contiguous."""
    rows, cols = T.shape[-2:]
    if T.stride(-1) != 1 and cols > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    ld = max(T.stride(-2), cols) if rows > 1 else max(cols, 1)
    return (1, ld, 0) if T.dim() == 2 else (T.shape[0], ld, T.stride(0))


def orthogonalize(G, steps=5, coefficients=QUINTIC, eps=1e-7, out=None, out_dtype=None,
                  workspace=None, stream=None):
    """G (rows x cols, or a batch of such matrices) orthogonalised by `steps`
    Newton-Schulz steps: every singular value towards 1.

    coefficients: (a, b, c) for all steps, or one such triple per step.  out:
    the result, of G's shape (it may be G itself), allocated as out_dtype (G's
    own type if None) when None.  The workspace comes from PyTorch's caching
    allocator unless given (dga_orthogonalize_workspace_size bytes)."""
    if G.dim() not in (2, 3):
        raise ValueError("G must be a matrix or a batch of matrices")
    if G.dtype not in _CODE:
        raise TypeError("G must be float32, bfloat16 or float16")
    if not G.is_cuda:
        raise ValueError("G must be a CUDA tensor")
    if out is None:
        out = torch.empty(G.shape, dtype=G.dtype if out_dtype is None else _TORCH[out_dtype], device=G.device)
    elif out.shape != G.shape or out.dtype not in _CODE or out.device != G.device:
        raise ValueError("out must be a float32, bfloat16 or float16 tensor of G's shape, on its device")
    flat = [float(c) for t in coefficients for c in t] if hasattr(coefficients[0], "__len__") \
        else [float(c) for c in coefficients] * steps
    if len(flat) != 3 * steps:
        raise ValueError(f"coefficients must be one (a, b, c), or {steps} of them")
    batch, ldg, stride_g = _layout(G, "G")
    _, ldo, stride_o = _layout(out, "out")
    rows, cols = G.shape[-2:]
    code = _CODE[out.dtype]
    need = dga_orthogonalize_workspace_size(code, batch, rows, cols)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=G.device)
    if stream is None:
        stream = torch.cuda.current_stream(G.device).cuda_stream
    st = lib().dga_orthogonalize(_CODE[G.dtype], code, batch, rows, cols, G.data_ptr(), ldg, stride_g,
                                 out.data_ptr(), ldo, stride_o, steps, (ctypes.c_float * len(flat))(*flat),
                                 eps, workspace.data_ptr() if workspace.numel() else None,
                                 workspace.numel() * workspace.element_size(), stream)
    if st != OK:
        raise DgaError(st, "dga_orthogonalize")
    return out
