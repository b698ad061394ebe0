"""Products of operands whose rows are a multiple of 16 bytes apart but do not
start on 16 bytes: views that leave out a first column."""
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tf32", [False, True])
@pytest.mark.parametrize("M", [1, 7, 16, 130, 600])
@pytest.mark.parametrize("which", ["A", "B", "AB"])
@pytest.mark.parametrize("transposed", [False, True])
def test_views_without_their_first_column(tf32, M, which, transposed):
    """Small integers: every sum is exact, whichever kernel and repack runs."""
    N, K, dtype = 200, 304, torch.float32 if tf32 else torch.bfloat16
    g = torch.Generator().manual_seed(M)

    def operand(rows, cols, off):
        base = torch.full((rows, (cols + 15) // 8 * 8), float("nan"), dtype=dtype)
        base[:, off:off + cols] = torch.randint(-3, 4, (rows, cols), generator=g).to(dtype)
        return base.cuda()[:, off:off + cols]

    A = operand(M, K, 1 if "A" in which else 0)
    B = operand(N, K, 1 if "B" in which else 0).t() if transposed else operand(K, N, 1 if "B" in which else 0)
    got = dga.gemm(A, B, tf32=tf32, out_dtype=dga.F32)
    assert torch.equal(got.double(), A.double() @ B.double())
    if not tf32 and transposed:
        W = B.t()
        assert torch.equal(dga.linear_forward(A, W).double(), (A.double() @ B.double()).bfloat16().double())
