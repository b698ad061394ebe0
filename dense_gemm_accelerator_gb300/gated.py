"""The gated feed-forward layer, H = act(X Wg^T + bg) * (X Wu^T + bu), and its
gradients: PyTorch-tensor forms of ``dga_gated`` and ``dga_gated_backward``
(include/dga.h has the formulas, roundings and errors).  The weight W holds the
gate's rows before the up projection's, [2 * hidden, in], and the bias likewise.
All work runs in the library's CUDA kernels on the current stream of the
tensors' device, or the one given; scratch and results come from PyTorch's
caching allocator, on the same stream.
"""
from __future__ import annotations

import functools

import torch

from . import F32, DgaError, _current_device, _elsewhere, _on_device, _raw_stream, lib
from .mx import _CODE, _rows_of, on_stream

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3, "sigmoid": 4}


# sizes of scratch, by shape and by the (current) device, whose number of SMs decides
# how far products are cut
@functools.lru_cache(maxsize=4096)
def _forward_workspace(device, code, M, F, K, ldx, ldw, save):
    return lib().dga_gated_workspace_size(code, M, F, K, ldx, ldw, save)


@functools.lru_cache(maxsize=4096)
def _backward_workspace(device, code, M, F, K, ldx, ldw):
    return lib().dga_gated_backward_workspace_size(code, M, F, K, ldx, ldw)


def activation_code(activation):
    code = ACTIVATIONS.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}")
    return code


def _check(T, name, dtype, device):
    if T.dtype is not dtype:
        raise TypeError(f"{name} must have the type of X")
    if T.device != device:
        raise ValueError(f"{name} must be on the device of X")


def vector(b, n, dtype, device):
    """The pointer of a bias of n values, or None."""
    if b is None:
        return None
    if b.dim() != 1 or b.numel() != n or (n > 1 and b.stride(0) != 1) or b.dtype is not dtype or b.device != device:
        raise ValueError(f"bias must be a contiguous vector of {n} values of the type and device of X")
    return b.data_ptr()


def result(T, rows, cols, dtype, device, name):
    """(an output, allocated where T is None, its leading dimension)."""
    if T is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), cols or 1
    if T.dim() != 2 or T.size(0) != rows or T.size(1) != cols or T.dtype is not dtype or T.device != device:
        raise ValueError(f"{name} must be a ({rows}, {cols}) tensor of the type and device of X")
    return T, _rows_of(T, name)[2]


def odd_where_off(ld, pointer):
    """A leading dimension as the size queries take it for a pointer off 16 bytes."""
    return ld if pointer % 16 == 0 else ld | 1


def scratch(workspace, d):
    """The bytes of a workspace that a caller gives (to the kernels, an address and these)."""
    if workspace.get_device() != d or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the device of X")
    return workspace.numel() * workspace.element_size()


def gated_forward(X, W, bias=None, activation="silu", save=False, H=None, P=None, workspace=None, stream=None):
    """H = act(g) * u with [g | u] = X @ W^T + bias, for X [batch, in], W [2 * hidden,
    in] and bias [2 * hidden] of one type (float32, bfloat16 or float16), row-major;
    activation: "silu", "gelu", "gelu_tanh", "relu" or "sigmoid".  Returns H [batch,
    hidden], or with save=True (H, P), P = [g | u] being what gated_backward reads.
    H, P and the workspace are allocated unless given; a P that is given is written."""
    if stream is not None:
        return on_stream(stream, X.device, gated_forward, X, W, bias, activation, save, H, P, workspace)
    dtype, act, d = X.dtype, activation_code(activation), X.get_device()
    code = _CODE.get(dtype)
    if code is None:
        raise TypeError("X must be float32, bfloat16 or float16")
    if d < 0:
        raise ValueError("X must be a CUDA tensor")
    if W.dtype is not dtype or W.get_device() != d:
        _check(W, "W", dtype, X.device)
    if d != _current_device():
        return _on_device(X.device, gated_forward, X, W, bias, activation, save, H, P, workspace)
    M, K, ldx = _rows_of(X, "X")
    N, k, ldw = _rows_of(W, "W")
    if k != K or N % 2:
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)} (an even number of rows of X's length)")
    F = N // 2
    if H is None:
        H, ldh = torch.empty((M, F), dtype=dtype, device=d), F or 1
    else:
        H, ldh = result(H, M, F, dtype, X.device, "H")
    save = save or P is not None
    p, ldp = None, 0
    if save:
        P, ldp = result(P, M, N, dtype, X.device, "P")
        p = P.data_ptr()
    x, w = X.data_ptr(), W.data_ptr()
    if workspace is None:
        have = 0
        if ldx % 8 or ldw % 8 or (x | w) % 16 or code == F32 or not K:  # else none is needed
            have = _forward_workspace(d, code, M, F, K, odd_where_off(ldx, x), odd_where_off(ldw, w), 1 if save else 0)
        if have:
            workspace = torch.empty(have, dtype=torch.uint8, device=d)
    else:
        have = scratch(workspace, d)
    st = lib().dga_gated(code, act, M, F, K, x, ldx, w, ldw, None if bias is None else vector(bias, N, dtype, X.device), H.data_ptr(),
                         ldh, p, ldp, workspace.data_ptr() if have else None, have, _raw_stream(d))
    if st:
        raise DgaError(st, "dga_gated")
    return (H, P) if save else H


def gated_backward(X, W, P, G, activation="silu", need_bias=False, need_x=True, need_w=True, dX=None, dW=None,
                   workspace=None, stream=None):
    """Gradients of the layer for H's gradient G [batch, hidden], from the inputs X and
    W and the pre-activations P [batch, 2 * hidden] that gated_forward saved, all of
    one type: (dX, dW, db), dX and dW in that type, db in float32; None for one that
    need_x, need_w or need_bias does not ask for."""
    if stream is not None:
        return on_stream(stream, X.device, gated_backward, X, W, P, G, activation, need_bias, need_x, need_w, dX, dW, workspace)
    dtype, dev = X.dtype, X.device
    code, act = _CODE.get(dtype), activation_code(activation)
    if code is None:
        raise TypeError("X must be float32, bfloat16 or float16")
    if not X.is_cuda:
        raise ValueError("X must be a CUDA tensor")
    for T, name in ((W, "W"), (P, "P"), (G, "G")):
        _check(T, name, dtype, dev)
    if _elsewhere(dev):
        return _on_device(dev, gated_backward, X, W, P, G, activation, need_bias, need_x, need_w, dX, dW, workspace)
    M, K, ldx = _rows_of(X, "X")
    N, k, ldw = _rows_of(W, "W")
    F = N // 2
    if k != K or N % 2 or tuple(P.shape) != (M, N) or tuple(G.shape) != (M, F):
        raise ValueError(f"shape mismatch: X {tuple(X.shape)}, W {tuple(W.shape)}, P {tuple(P.shape)}, G {tuple(G.shape)}")
    ldp, ldg = _rows_of(P, "P")[2], _rows_of(G, "G")[2]
    x, w = X.data_ptr(), W.data_ptr()
    db = torch.empty(N, dtype=torch.float32, device=dev) if need_bias else None
    dx = dw = None
    lddx = lddw = 0
    if need_x:
        dX, lddx = result(dX, M, K, dtype, dev, "dX")
        dx = dX.data_ptr()
    if need_w:
        dW, lddw = result(dW, N, K, dtype, dev, "dW")
        dw = dW.data_ptr()
    if workspace is None:
        have = _backward_workspace(dev.index, code, M, F, K, odd_where_off(ldx, x), odd_where_off(ldw, w))
        if have:
            workspace = torch.empty(have, dtype=torch.uint8, device=dev)
    else:
        have = scratch(workspace, dev.index)
    st = lib().dga_gated_backward(code, act, M, F, K, x, ldx, w, ldw, P.data_ptr(), ldp, G.data_ptr(), ldg, dx, lddx, dw,
                                  lddw, db.data_ptr() if need_bias else None, workspace.data_ptr() if have else None, have,
                                  _raw_stream(dev.index))
    if st:
        raise DgaError(st, "dga_gated_backward")
    return (dX if need_x else None), (dW if need_w else None), db
