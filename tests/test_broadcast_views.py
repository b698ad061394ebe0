"""Broadcast and overlapping views: their rows start less than a row's length
apart, which a leading dimension cannot say.  They are refused, whichever
argument they are, and never read or written as if they were apart."""
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from dense_gemm_accelerator_gb300 import muon, mx


def _views(rows, cols, device="cpu"):
    """Rows all the same, columns all the same, rows that overlap, one value."""
    memory = torch.arange(1.0, 1.0 + rows * cols, device=device)
    return [memory[:cols].expand(rows, cols), memory[:rows, None].expand(rows, cols),
            memory.as_strided((rows, cols), (cols - 1, 1)), memory[:1].expand(rows, cols)]


def _gradient_of_a_batch_sum(rows, cols, device="cpu"):
    """What autograd hands to a layer whose output is summed over the batch."""
    y = torch.zeros(rows, cols, device=device, requires_grad=True)
    seen = []
    z = y * 1.0
    z.register_hook(seen.append)
    z.sum(0).backward(torch.arange(1.0, cols + 1.0, device=device))
    return seen[0]


def test_a_batch_sums_gradient_is_such_a_view():
    assert _gradient_of_a_batch_sum(4, 5).stride() == (0, 1)


def test_rows_of():
    for v in _views(4, 5) + [_gradient_of_a_batch_sum(4, 5)]:
        with pytest.raises(ValueError):
            mx._rows_of(v, "X")
        with pytest.raises(ValueError):
            mx._rows_of(v.t(), "X")
    column = torch.ones(1).expand(4, 1)
    with pytest.raises(ValueError, match="overlap"):
        mx._rows_of(column, "X")


def test_layout_of_updates():
    for v in _views(4, 5) + [torch.ones(1).expand(4, 1)]:
        with pytest.raises(ValueError):
            muon._layout(v, "G")
        with pytest.raises(ValueError):
            muon._layout(v.expand(3, *v.shape), "G")


def test_layout_of_gemm_operands():
    x = torch.empty(4, 5)
    for v in _views(4, 5) + [torch.ones(1).expand(4, 1)]:
        with pytest.raises(ValueError):
            dga._layout_of(v, "A")
        with pytest.raises(ValueError):
            dga._layout_of(v.t(), "A")
    for v in _views(4, 5):
        with pytest.raises(ValueError):
            dga.operand_layout(v, torch.empty(5, 5), x)
        with pytest.raises(ValueError):
            dga.operand_layout(x, v.t(), torch.empty(4, 4))
        with pytest.raises(ValueError):
            dga.operand_layout(x, torch.empty(5, 5), v)
        with pytest.raises(ValueError):
            dga.sum_rows(v)


def test_lines_apart_are_taken_as_before():
    x = torch.empty(6, 8)
    assert mx._rows_of(x, "X") == (6, 8, 8)
    assert mx._rows_of(x[:, 1:4], "X") == (6, 3, 8)
    assert mx._rows_of(x[:, :1], "X") == (6, 1, 8)
    # one row: its stride says nothing
    assert mx._rows_of(x[:1].expand(1, 8), "X") == (1, 8, 8)
    assert mx._rows_of(torch.empty(8).as_strided((1, 8), (0, 1)), "X") == (1, 8, 8)
    assert mx._rows_of(torch.empty(5, 0), "X") == (5, 0, 1)
    assert muon._layout(x, "G") == (1, 6, 8, 8, 0)
    assert muon._layout(torch.empty(8).as_strided((1, 8), (0, 1)), "G") == (1, 1, 8, 8, 0)
    assert dga._layout_of(torch.empty(8).as_strided((1, 8), (0, 1)), "A") == (dga.ROW_MAJOR, 8)
    assert dga._layout_of(torch.empty(8).as_strided((8, 1), (1, 0)), "A") == (dga.ROW_MAJOR, 1)
    assert dga._layout_of(torch.empty(5, 0), "A") == (dga.ROW_MAJOR, 1)
    # matrices of a batch may be the same one
    assert muon._layout(x.expand(3, 6, 8), "G") == (3, 6, 8, 8, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [dga.MXFP4, dga.NVFP4])
@pytest.mark.parametrize("rows", [4, 40, 300])
def test_refused_by_the_4_bit_calls(fmt, rows):
    cols = 64
    x = torch.ones(rows, cols, device="cuda")
    w = torch.ones(cols, cols, device="cuda")
    W = dga.mx_quantize(w, fmt)
    q = dga.mx_quantize(x, fmt)
    for v in _views(rows, cols, "cuda") + [_gradient_of_a_batch_sum(rows, cols, "cuda")]:
        for call in (lambda: dga.mx_quantize(v, fmt), lambda: dga.mx_quantize(v, fmt, transpose=True),
                     lambda: dga.mx_linear_forward(v, W), lambda: dga.mx_linear_forward(x, W, Y=v),
                     lambda: dga.mx_gemm(q, W, v), lambda: dga.mx_linear_backward(v, w, x, fmt),
                     lambda: dga.mx_linear_backward(x, w, v, fmt)):
            with pytest.raises(ValueError):
                call()
    with pytest.raises(ValueError):
        dga.mx_linear_backward(x, w[:1].expand(cols, cols), x, fmt)
    # its copy is another matter
    g = _gradient_of_a_batch_sum(rows, cols, "cuda")
    dX, dW, db = dga.mx_linear_backward(x, w, g.contiguous(), fmt)
    assert torch.equal(db, g.double().sum(0).float())
    assert dX.shape == x.shape and dW.shape == w.shape


@pytest.mark.gpu
def test_refused_by_the_orthogonalisation():
    G = torch.ones(4, 5, device="cuda")
    for v in _views(4, 5, "cuda"):
        with pytest.raises(ValueError):
            dga.orthogonalize(v)
        with pytest.raises(ValueError):
            dga.orthogonalize(G, out=v)
    same = torch.randn(30, 50, generator=torch.Generator().manual_seed(1)).cuda()
    got = dga.orthogonalize(same.expand(3, 30, 50))
    assert all(torch.equal(got[i], dga.orthogonalize(same)) for i in range(3))


@pytest.mark.gpu
def test_refused_by_the_products():
    rows, cols = 20, 64
    x, w = torch.ones(rows, cols, device="cuda"), torch.ones(cols, cols, device="cuda")
    for v in _views(rows, cols, "cuda") + [_gradient_of_a_batch_sum(rows, cols, "cuda")]:
        for call in (lambda: dga.gemm(v, w), lambda: dga.gemm(v.t(), x), lambda: dga.gemm(w, v.t()), lambda: dga.gemm(x, w, v),
                     lambda: dga.sum_rows(v), lambda: dga.linear_forward(v, w), lambda: dga.linear_forward(x, w, Y=v),
                     lambda: dga.linear_backward(x, w, v), lambda: dga.linear_backward(v, w, x)):
            with pytest.raises(ValueError):
                call()
    dX, dW, db = dga.linear_backward(x, w, _gradient_of_a_batch_sum(rows, cols, "cuda").contiguous())
    assert torch.equal(db, rows * torch.arange(1.0, cols + 1, device="cuda"))
