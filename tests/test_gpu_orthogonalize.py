"""The Newton-Schulz orthogonalisation on the GPU against the formula in fp64."""
import numpy as np
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga

pytestmark = pytest.mark.gpu

# Relative 2-norm tolerances, from a simulation of the kernels' roundings (the
# operands' 11 or 22 bits, fp32 sums) against fp64: at most 1.7e-3 from the
# products' 11-bit operands and 1.7e-3 from the output's own rounding to bf16
# (2e-4 to fp16); 9e-6 with 22-bit operands on momentum of low rank over noise
# of a twentieth its size, 2.6e-5 over noise of a thousandth.  Doubled.
TOL = {torch.bfloat16: 5e-3, torch.float16: 6e-4, torch.float32: 2e-5}
TOL_STRONG = {torch.bfloat16: 5e-3, torch.float16: 6e-4, torch.float32: 6e-5}


def _formula(G, steps=5, coefficients=None, eps=1e-7):
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    X = X / (torch.linalg.matrix_norm(X, keepdim=True) + eps)
    for s in range(steps):
        a, b, c = (coefficients or [dga.QUINTIC] * steps)[s]
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if tall else X


def _rel(got, want):
    d = (got.cpu().double() - want).flatten(-2).norm(dim=-1)
    return float((d / want.flatten(-2).norm(dim=-1)).max())


def _ok():
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


def _momentum(shape, seed, rank=4, noise=0.05):
    g = torch.Generator().manual_seed(seed)
    *b, m, n = shape
    low = torch.randn(*b, m, rank, generator=g) @ torch.randn(*b, rank, n, generator=g)
    return low + noise * torch.randn(*b, m, n, generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (64, 64), (65, 63), (100, 300), (300, 100), (256, 256),
                                   (257, 260), (513, 129), (515, 1030), (700, 640), (3, 100, 65), (5, 130, 257),
                                   (40, 64, 64), (12, 300, 270), (1, 1100, 700), (128, 128), (127, 640), (1500, 100),
                                   (120, 2048), (128, 2049), (80, 90, 200), (30, 500, 64), (3, 33, 1700)])
def test_against_the_formula(dtype, shape):
    g = torch.Generator().manual_seed(sum(shape))
    for G, tol in ((torch.randn(*shape, generator=g), TOL), (1e-3 * _momentum(shape, 1), TOL),
                   (_momentum(shape, 2, noise=1e-3), TOL_STRONG)):
        G = G.to(dtype)
        got = dga.orthogonalize(G.cuda())
        _ok()
        assert got.dtype == dtype and got.shape == G.shape
        assert _rel(got, _formula(G)) <= tol[dtype]


@pytest.mark.parametrize("shape", [(2100, 2200), (2500, 2100)])
def test_large_enough_for_cta_pairs(shape):
    G = _momentum(shape, 3)
    for dtype in (torch.float32, torch.bfloat16):
        x = G.to(dtype)
        got = dga.orthogonalize(x.cuda())
        _ok()
        want = _formula(x.cuda()).cpu()
        assert _rel(got, want) <= TOL[dtype]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(12, 515, 1030), (12, 1030, 515), (20, 259, 270), (9, 770, 580)])
def test_batches_on_cta_pairs_with_thin_last_tiles(dtype, shape):
    """256 x 256 tiles of which the last hold a few rows or columns, several
    rounds of them, into results whose rows TMA can and cannot store."""
    G = _momentum(shape, 11).to(dtype).cuda()
    want = _formula(G).cpu()
    got = dga.orthogonalize(G)
    frame = torch.full((shape[0], shape[1] + 2, shape[2] + 5), 7.0, dtype=dtype, device="cuda")
    dga.orthogonalize(G, out=frame[:, 1:-1, 3:-2])
    _ok()
    assert _rel(got, want) <= TOL[dtype]
    assert torch.equal(frame[:, 1:-1, 3:-2], got)
    frame[:, 1:-1, 3:-2] = 7.0
    assert (frame == 7.0).all(), "written outside the result"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(14, 515, 700), (26, 300, 310), (3, 1025, 2050)])
def test_a_last_round_of_few_tiles(dtype, shape):
    """Tile counts just past a whole number of rounds, symmetric products among them."""
    G = _momentum(shape, 13).to(dtype).cuda()
    got = dga.orthogonalize(G)
    _ok()
    assert _rel(got, _formula(G).cpu()) <= TOL[dtype]
    assert torch.equal(got, dga.orthogonalize(G))


def test_offsets_past_32_bits():
    """A 140 x 16,000,000 update (2.24e9 values): the columns at both ends, from
    fp64 products."""
    m, n = 140, 16_000_000
    g = torch.Generator(device="cuda").manual_seed(12)
    G = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    for c in range(0, n, 1_000_000):
        G[:, c:c + 1_000_000] = torch.randn(m, 1_000_000, device="cuda", generator=g)
    got = dga.orthogonalize(G, steps=1, coefficients=(1.5, -0.5, 0.0))
    _ok()
    A = torch.zeros(m, m, dtype=torch.float64, device="cuda")
    for c in range(0, n, 1_000_000):
        x = G[:, c:c + 1_000_000].double()
        A += x @ x.mT
    norm2 = float(A.diagonal().sum())
    for c in (0, n // 2 - 50, n - 100):
        x = G[:, c:c + 100].double() / norm2 ** 0.5
        want = 1.5 * x - 0.5 * (A / norm2) @ x
        assert float((got[:, c:c + 100].double() - want).norm() / want.norm()) <= TOL[torch.bfloat16]


def test_types_steps_and_coefficients():
    G = _momentum((90, 200), 4)
    cases = [(3, dga.QUINTIC), (1, (1.5, -0.5, 0.0)), (4, [(3.0, -4.0, 1.6), (2.5, -3.0, 1.2), (2.0, -1.6, 0.6), (1.875, -1.25, 0.375)])]
    for steps, co in cases:
        per = co if isinstance(co, list) else [co] * steps
        for src, dst in ((torch.float32, dga.BF16), (torch.bfloat16, dga.F32), (torch.float16, dga.F32)):
            x = G.to(src)
            got = dga.orthogonalize(x.cuda(), steps=steps, coefficients=co, out_dtype=dst)
            assert _rel(got, _formula(x, steps, per)) <= (TOL[torch.float32] if dst == dga.F32 else TOL[torch.bfloat16])
    x = G * 1e-6
    assert _rel(dga.orthogonalize(x.cuda(), eps=1e-3), _formula(x, eps=1e-3)) <= TOL[torch.float32]


def test_singular_values_near_one():
    s = torch.linalg.svdvals(dga.orthogonalize(torch.randn(400, 900, generator=torch.Generator().manual_seed(1)).cuda()).double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


def test_strides_out_and_in_place():
    base = _momentum((3, 70, 150), 5)
    d = base.cuda()
    for view, out in ((d[:, 3:60, 1:131], None), (d[:, ::2, :], None), (d[1], torch.empty(70, 160, device="cuda")[:, 5:155]),
                      (d[:2, :, :70], torch.full((2, 75, 90), 7.0, device="cuda")[:, 2:72, 3:73])):
        got = dga.orthogonalize(view, out=out)
        assert _rel(got, _formula(view.cpu())) <= TOL[torch.float32]
    frame = torch.full((2, 75, 90), 7.0, device="cuda")
    dga.orthogonalize(d[:2, :, :70], out=frame[:, 2:72, 3:73])
    frame[:, 2:72, 3:73] = 7.0
    assert (frame == 7.0).all(), "written outside the result"
    x = d.clone()
    assert dga.orthogonalize(x, out=x) is x
    assert _rel(x, _formula(base)) <= TOL[torch.float32]


def test_zero_and_not_finite_matrices_stay_apart():
    G = torch.randn(4, 130, 140, generator=torch.Generator().manual_seed(6))
    G[1] = 0.0
    G[2, 5, 6] = float("nan")
    for dtype in (torch.float32, torch.bfloat16):
        x = G.to(dtype)
        got = dga.orthogonalize(x.cuda()).cpu()
        _ok()
        want = _formula(x)
        assert (got[1] == 0).all() and torch.isnan(got[2]).all()
        for i in (0, 3):
            assert _rel(got[i], want[i]) <= TOL[dtype]


def test_repeats_bit_for_bit_on_streams_and_in_a_graph():
    for shape in ((200, 300), (700, 900)):
        G = _momentum(shape, 7).cuda()
        want = dga.orthogonalize(G)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = dga.orthogonalize(G)
        s.synchronize()
        assert torch.equal(got, want)
        x = G.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = dga.orthogonalize(x)
        x.copy_(G.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, dga.orthogonalize(G.flip(0).contiguous()))


def test_empty_and_refusals():
    assert dga.orthogonalize(torch.empty(0, 5, device="cuda")).shape == (0, 5)
    assert dga.orthogonalize(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    G = torch.ones(4, 5, device="cuda")
    with pytest.raises(ValueError):
        dga.orthogonalize(torch.ones(5, device="cuda"))
    with pytest.raises(TypeError):
        dga.orthogonalize(torch.ones(4, 5, device="cuda", dtype=torch.float64))
    with pytest.raises(ValueError):
        dga.orthogonalize(torch.ones(4, 5))
    with pytest.raises(ValueError):
        dga.orthogonalize(G.t())
    with pytest.raises(ValueError):
        dga.orthogonalize(G, coefficients=[(1.0, 2.0, 3.0)] * 2)
    with pytest.raises(ValueError):
        dga.orthogonalize(G, out=torch.empty(4, 6, device="cuda"))
    with pytest.raises(dga.DgaError):
        dga.orthogonalize(G, steps=0)
    with pytest.raises(dga.DgaError):
        dga.orthogonalize(G, eps=-1.0)
    with pytest.raises(dga.DgaError):
        dga.orthogonalize(G, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
