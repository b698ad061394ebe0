"""Products on 4-bit weights at the ends of X's range, at weights whose scale table is past
the few-row kernel's shared memory, and with the roundings that the header promises."""
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import gated_reference as ref
from tests.test_gpu_q4 import HALVES, _values, _weight, _x


def _check(X, Q, bias=None):
    """Within fp32's sums of unrounded weights, and the result's rounding."""
    v, off = ref.product(X, _values(Q), bias)
    ref.within(dga.q4_linear_forward(X, Q, bias), v, off + ref.rounding(v, X.dtype) * (1 + 2.0 ** -7))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 9, 17, 32, 40, 100, 1100])
def test_the_largest_activations(M, group, dtype):
    """Rows of the type's lowest or largest value, of both in turn, and with one such value:
    scales of 2^-12, with which every value is exact in either type and no result, nor
    a part of its sum, passes the type's range (K = 256: 256 * 15 * 2^-12 < 1)."""
    N, K = 200, 256
    top = torch.finfo(dtype).max
    for zeros in (False, True):
        Q = _weight(N, K, group, zeros, dtype, M)
        Q.scales.fill_(2.0 ** -12)
        X = _x(M, K, dtype, M)
        for row, value in ((0, -top), (M // 2, top), (M - 1, -top)):
            X[row] = value
        if M > 3:
            X[1, 1::2], X[1, 0::2] = top, -top
            X[3, 77] = -top
        _check(X, Q)
    Q = _weight(2 * N, K, group, True, dtype, M)
    Q.scales[:N].fill_(2.0 ** -12)
    Q.scales[N:].fill_(2.0 ** -14 / top)  # up: up to 1/4
    H = dga.q4_gated_forward(X, Q, activation="relu")
    P, off = ref.product(X, _values(Q))
    ref.within(H, *ref.gated_of(P, off, "relu", dtype))
    assert bool(torch.isfinite(H).all())
