"""The gated layer with relu on small whole numbers, whose sums fp32 holds exactly: long
rows, many rows, and what infinities and NaN reach."""
import math

import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import gated_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _whole(g, *shape, most=1):
    return torch.randint(-most, most + 1, shape, device="cuda", generator=g).float()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", [(1, 40, 100003), (16, 3, 70000), (17, 40, 70001), (130, 5, 33000), (300, 520, 9001), (1, 20000, 64)])
def test_forward(M, F, K, dtype):
    """Sums below 2^24 are exact in any order; H is the fp32 product of two of them, rounded."""
    g = torch.Generator(device="cuda").manual_seed(M + F)
    X, W, b = _whole(g, M, K), _whole(g, 2 * F, K), _whole(g, 2 * F, most=3)
    P = X.double() @ W.double().t() + b.double()
    assert float(P.abs().max()) < 2 ** 24
    H, got = dga.gated_forward(X.to(dtype), W.to(dtype), b.to(dtype), activation="relu", save=True)
    assert torch.equal(got, P.to(dtype))
    assert torch.equal(H, (P[:, :F].clamp(min=0) * P[:, F:]).float().to(dtype))
    assert torch.equal(dga.gated_forward(X.to(dtype), W.to(dtype), b.to(dtype), activation="relu"), H)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", [(70001, 20, 24), (33333, 3, 130), (5, 40000, 9), (1, 12000, 300), (1200, 257, 515)])
def test_backward(M, F, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    X, W, P, G = _whole(g, M, K), _whole(g, 2 * F, K), _whole(g, M, 2 * F, most=3), _whole(g, M, F, most=2)
    gate, up = P[:, :F], P[:, F:]
    dP = torch.cat([G * up * (gate > 0), G * gate.clamp(min=0)], 1).double()
    want = dP @ W.double(), dP.t() @ X.double(), dP.sum(0)
    assert max(float(w.abs().max()) for w in want) < 2 ** 24
    got = dga.gated_backward(X.to(dtype), W.to(dtype), P.to(dtype), G.to(dtype), activation="relu", need_bias=True)
    assert torch.equal(got[0], want[0].to(dtype)) and torch.equal(got[1], want[1].to(dtype)) and torch.equal(got[2], want[2].float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_infinities_stay_in_their_rows_and_columns(M, dtype):
    """A token with an infinity and a NaN, and a weight row with a NaN: every output of
    that token, or of that column, and nothing else; rows of zeros (padding) give zeros."""
    F, K = 72, 100
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn(M, K, device="cuda", generator=g).to(dtype)
    W = (torch.randn(2 * F, K, device="cuda", generator=g) / 10).to(dtype)
    if M > 2:
        X[M - 1] = 0
    for name in ref.ACTS:
        want = dga.gated_forward(X, W, activation=name)
        if M > 2:
            assert not want[M - 1].any()
        Xb = X.clone()
        Xb[0, 17], Xb[0, 90] = math.inf, math.nan
        got = dga.gated_forward(Xb, W, activation=name)
        assert bool(torch.isnan(got[0]).all()) and torch.equal(got[1:], want[1:])
        for row, column in ((5, 5), (F + 11, 11)):
            Wb = W.clone()
            Wb[row, 3] = math.nan
            got = dga.gated_forward(X, Wb, activation=name)
            keep = torch.arange(F, device="cuda") != column
            assert bool(torch.isnan(got[:, column]).all()) and torch.equal(got[:, keep], want[:, keep])
