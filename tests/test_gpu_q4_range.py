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


# ---- weights that are not rounded ---------------------------------------------------------


def _on(device, M, N, K, group, zeros, dtype, seed):
    """X and a weight whose values (q - z) s do not fit dtype."""
    g = torch.Generator().manual_seed(seed)
    width, groups = (K + 31) // 32 * 16, -(-K // group)
    codes = torch.randint(0, 256, (N, width), dtype=torch.uint8, generator=g)
    scales = (0.02 * torch.randn(N, groups, generator=g)).to(dtype)
    z = torch.randint(0, 16, (N, groups), dtype=torch.uint8, generator=g).to(device) if zeros else None
    return torch.randn(M, K, generator=g).to(dtype).to(device), dga.Q4Tensor(K, group, codes.to(device), scales.to(device), z)


@pytest.mark.parametrize("dtype", HALVES)
def test_the_bound_sees_rounded_weights(dtype):
    """On the CPU: exact sums of weights rounded to dtype are outside the bound of _check."""
    X, Q = _on("cpu", 20, 200, 256, 64, True, dtype, 1)
    V = _values(Q)
    v, off = ref.product(X, V)
    for W, fits in ((V, True), (V.to(dtype).double(), False)):
        got = (X.double() @ W.t()).to(dtype)
        if fits:
            ref.within(got, v, off + ref.rounding(v, dtype))
        else:
            with pytest.raises(AssertionError):
                ref.within(got, v, off + ref.rounding(v, dtype) * (1 + 2.0 ** -7))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 200, 256), (16, 200, 256), (17, 200, 256), (24, 9000, 520), (32, 8200, 512), (33, 200, 256), (48, 16384, 256),
                                   (64, 4096, 200), (64, 130, 264)])
def test_few_rows_take_the_weights_unrounded(M, N, K, group, dtype):
    """Up to 32 rows, and 64 where N K is at most 2^22."""
    assert M <= 32 or N * K <= 1 << 22
    for zeros in (False, True):
        X, Q = _on("cuda", M, N, K, group, zeros, dtype, M + N)
        _check(X, Q, torch.randn(N, device="cuda").to(dtype) if zeros else None)
        F = N // 2
        P, off = ref.product(X, _values(Q))
        ref.within(dga.q4_gated_forward(X, Q, activation="relu"), *ref.gated_of(P, off, "relu", dtype))


# ---- long K -------------------------------------------------------------------------------


def _whole(M, N, K, group, dtype, seed):
    """X of -1, 0 and 1 and scales of 1 and 2: every sum is a whole number below 2^22."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q = _weight(N, K, group, True, dtype, seed)
    Q.scales.copy_(torch.randint(1, 3, Q.scales.shape, device="cuda", generator=g))
    return torch.randint(-1, 2, (M, K), device="cuda", generator=g).to(dtype), Q


# a table of scales of one, two or four tiles of 16 weight rows that does not fit the few-row kernel's
# shared memory (groups of 32: from K = 51200, 25600, 12800 on; of 64 from the same, of 128 from twice
# that), and K as long for the other kernels
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("M,N,K,group", [(1, 5000, 16648, 32), (13, 5000, 14000, 64), (30, 4900, 28672, 128), (5, 3000, 28680, 32), (20, 3000, 26001, 64),
                                         (3, 1000, 52000, 32), (9, 500, 51333, 64), (40, 60, 66000, 64), (64, 130, 14000, 32), (64, 20, 104000, 128),
                                         (33, 300, 52000, 32), (100, 200, 30000, 128), (300, 130, 20001, 64), (1030, 64, 16640, 32)])
def test_long_rows(M, N, K, group, dtype):
    X, Q = _whole(M, N, K, group, dtype, M + K)
    P = X.double() @ _values(Q).t()
    assert float(P.abs().max()) < 2 ** 22
    got = dga.q4_linear_forward(X, Q)
    assert torch.equal(got, P.to(dtype))
    F = N // 2
    H = dga.q4_gated_forward(X, Q, activation="relu")
    assert torch.equal(H, (P[:, :F].clamp(min=0) * P[:, F:]).float().to(dtype))  # the fp32 product is rounded, then H
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK
