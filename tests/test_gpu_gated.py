"""The gated feed-forward layer and its gradients on the GPU against their
formulas in fp64 (tests/gated_reference.py)."""
import math

import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import gated_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# one value; below, at and past a vector, a tile of each kernel and the few-row kernel's rows
SIZES = [(1, 1, 1), (1, 8, 16), (2, 3, 5), (5, 64, 520), (13, 100, 264), (16, 250, 1000), (17, 16, 8), (40, 130, 100), (128, 128, 256),
         (129, 257, 130), (260, 515, 333), (300, 384, 64)]


def _inputs(M, F, K, dtype, seed, bias=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    X = (r(M, K) * torch.exp(0.5 * r(K))).to(dtype)
    W = (r(2 * F, K) * (2 / math.sqrt(K))).to(dtype)
    return X, W, r(2 * F).to(dtype) if bias else None


def _status_ok():
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


def _check_forward(X, W, b, name, H, P=None):
    want, eh, p, ep = ref.gated(X, W, b, name)
    ref.within(H, want, eh, "H")
    if P is not None:
        ref.within(P, p, ep, "P")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", SIZES)
def test_forward(M, F, K, dtype):
    for i, name in enumerate(ref.ACTS):
        X, W, b = _inputs(M, F, K, dtype, M * 7 + F + i, bias=i % 2 == 0)
        H = dga.gated_forward(X, W, b, activation=name)
        _check_forward(X, W, b, name, H)
        H2, P = dga.gated_forward(X, W, b, activation=name, save=True)
        assert H.dtype is dtype and P.dtype is dtype
        _check_forward(X, W, b, name, H2, P)
    _status_ok()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", SIZES)
def test_backward(M, F, K, dtype):
    for i, name in enumerate(ref.ACTS):
        X, W, _ = _inputs(M, F, K, dtype, M + F * 3 + i)
        g = torch.Generator(device="cuda").manual_seed(i)
        P = (2 * torch.randn(M, 2 * F, device="cuda", generator=g)).to(dtype)
        G = torch.randn(M, F, device="cuda", generator=g).to(dtype)
        dX, dW, db = dga.gated_backward(X, W, P, G, activation=name, need_bias=True)
        want = ref.gated_grads(X, W, P, G, name)
        for got, key in ((dX, "dX"), (dW, "dW"), (db, "db")):
            ref.within(got, *want[key], (key, name))
        assert dX.dtype is dtype and dW.dtype is dtype and db.dtype is torch.float32
    _status_ok()


@pytest.mark.parametrize("name", ref.ACTS)
def test_gradient_against_differences(name):
    """The loss sum(C * H) along a random direction, differenced in fp64 (step 1e-5: off by
    its square times the third derivative, below 1e-8 of these sums); the fp32 gradients'
    own errors are at most 1e-4 of the sums of magnitudes."""
    M, F, K = 7, 12, 20
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    X, W, b, C = r(M, K), r(2 * F, K) / 4, r(2 * F), r(M, F)
    _, P = dga.gated_forward(X, W, b, activation=name, save=True)
    if name == "relu":  # keep every sum away from the corner
        assert float(P[:, :F].abs().min()) > 1e-3
    dX, dW, db = dga.gated_backward(X, W, P, C, activation=name, need_bias=True)
    dx, dw, dv = r(M, K).double(), r(2 * F, K).double(), r(2 * F).double()

    def loss(h):
        p = (X.double() + h * dx) @ (W.double() + h * dw).t() + b.double() + h * dv
        return float((C.double() * ref.act(p[:, :F], name) * p[:, F:]).sum())

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    parts = [dX.double() * dx, dW.double() * dw, db.double() * dv]
    got = float(sum(p.sum() for p in parts))
    assert abs(got - slope) <= 1e-4 * float(sum(p.abs().sum() for p in parts))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [3, 100, 300])
def test_views_and_what_lies_around_the_results(M, dtype):
    """Padded leading dimensions, bases off 16 bytes, outputs inside larger arrays whose
    other values stay as they were."""
    F, K = 72, 100
    for off, pad in ((0, 0), (0, 8), (1, 3), (4, 4), (3, 0)):
        X, W, b = _inputs(M, F, K, dtype, 11 + off)

        def held(t, rows, cols):
            base = torch.full((rows * (cols + pad) + off + 5,), 7.0, dtype=dtype, device="cuda")
            v = base[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
            if t is not None:
                v.copy_(t)
            return base, v

        _, Xv = held(X, M, K)
        _, Wv = held(W, 2 * F, K)
        hb, H = held(None, M, F)
        pb, P = held(None, M, 2 * F)
        got, gp = dga.gated_forward(Xv, Wv, b, H=H, P=P)
        assert got is H and gp is P
        _check_forward(X, W, b, "silu", H, P)
        G = torch.randn(M, F, device="cuda").to(dtype)
        _, Gv = held(G, M, F)
        xb, dX = held(None, M, K)
        wb, dW = held(None, 2 * F, K)
        db = dga.gated_backward(Xv, Wv, P, Gv, need_bias=True, dX=dX, dW=dW)[2]
        want = ref.gated_grads(X, W, P, G, "silu")
        for t, key in ((dX, "dX"), (dW, "dW"), (db, "db")):
            ref.within(t, *want[key], key)
        for base, v in ((hb, H), (pb, P), (xb, dX), (wb, dW)):
            v.fill_(7.0)
            assert bool((base == 7.0).all())


def test_far_values_and_infinities():
    """Gates far from 0, infinities and NaN: what the formulas give in fp32."""
    g = torch.tensor([0.0, -0.0, 1e-30, 20.0, -20.0, 88.0, -88.0, 200.0, -200.0, 6e4, -6e4, math.inf, math.nan], device="cuda")
    for dtype in TYPES:
        for name in ref.ACTS:
            for M in (1, 200):
                F = g.numel()
                X = torch.ones(M, 1, device="cuda", dtype=dtype)
                W = torch.cat([g, torch.full((F,), 2.0, device="cuda")]).to(dtype)[:, None].contiguous()
                H, P = dga.gated_forward(X, W, activation=name, save=True)
                v = W[:F, 0].double()
                want = (ref.act(v, name) * 2).float().expand(M, F)
                got = H.float()
                assert torch.equal(torch.isnan(got), torch.isnan(want)), (name, dtype)
                fine = torch.isfinite(want)
                tol = 2 * ref.ACT_ERR * torch.clamp(v.abs(), min=1.0) + ref.rounding(want.double(), dtype)
                over = want.abs() > torch.finfo(dtype).max
                ok = ((got.double() - want.double()).abs() <= tol) | ~fine | over
                assert bool(ok.all()), (name, dtype, M)
                assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
                # the slopes of what is finite
                G = torch.ones(M, F, device="cuda", dtype=dtype)
                dX, dW, db = dga.gated_backward(X, W, P, G, activation=name, need_bias=True)
                pg = P[0, :F].double()
                ok = torch.isfinite(pg)
                want = M * 2 * ref.slope(pg, name)[ok]
                want = torch.where(torch.isnan(want), (pg[ok] > 0).double() * M * 2, want)
                assert bool(((db[:F][ok].double() - want).abs() <= M * 2 * (ref.ACT_ERR * torch.clamp(pg[ok].abs(), min=1.0))).all()), (name, dtype)


def test_empty_sizes():
    for dtype in TYPES:
        Z = lambda *s: torch.zeros(*s, device="cuda", dtype=dtype)  # noqa: E731
        assert dga.gated_forward(Z(0, 4), Z(6, 4)).shape == (0, 3)
        assert dga.gated_forward(Z(5, 4), Z(0, 4)).shape == (5, 0)
        b = torch.tensor([1.0, -2.0, 3.0, 0.5], device="cuda").to(dtype)
        for M in (1, 20, 200):
            H, P = dga.gated_forward(Z(M, 0), Z(4, 0), b, activation="relu", save=True)
            assert torch.equal(P, b.expand(M, 4)) and torch.equal(H.float(), torch.tensor([3.0, 0.0], device="cuda").expand(M, 2))
        dX, dW, db = dga.gated_backward(Z(0, 4), Z(6, 4), Z(0, 6), Z(0, 3), need_bias=True)
        assert dX.shape == (0, 4) and not dW.any() and not db.any()
        dX, dW, db = dga.gated_backward(Z(5, 4) + 1, Z(0, 4), Z(5, 0), Z(5, 0), need_bias=True)
        assert dX.shape == (5, 4) and not dX.any() and dW.shape == (0, 4) and db.shape == (0,)
        dX, dW, db = dga.gated_backward(Z(5, 0), Z(6, 0), Z(5, 6) + 1, Z(5, 3) + 1, need_bias=True, activation="relu")
        assert dX.shape == (5, 0) and dW.shape == (6, 0) and torch.equal(db, torch.full((6,), 5.0, device="cuda"))


def test_gradients_that_are_not_wanted():
    X, W, _ = _inputs(50, 30, 40, torch.bfloat16, 1)
    P, G = (torch.randn(50, n, device="cuda").bfloat16() for n in (60, 30))
    dX, dW, db = dga.gated_backward(X, W, P, G, need_bias=True)
    for need_x, need_w, need_b in ((True, False, False), (False, True, True), (False, False, True)):
        a, b, c = dga.gated_backward(X, W, P, G, need_x=need_x, need_w=need_w, need_bias=need_b)
        for got, want, need in ((a, dX, need_x), (b, dW, need_w), (c, db, need_b)):
            assert torch.equal(got, want) if need else got is None


@pytest.mark.parametrize("dtype,M", [(torch.bfloat16, 4), (torch.bfloat16, 100), (torch.float16, 600), (torch.float32, 300)])
def test_graph_streams_and_repeats(dtype, M):
    """Captured and replayed, on another stream, on two streams at once, and again: the same bits."""
    F, K = 384, 256
    X, W, b = _inputs(M, F, K, dtype, 3)
    G = torch.randn(M, F, device="cuda").to(dtype)

    def step(stream=None):
        H, P = dga.gated_forward(X, W, b, activation="gelu", save=True, stream=stream)
        return (H, P, *dga.gated_backward(X, W, P, G, activation="gelu", need_bias=True, stream=stream))

    want = step()
    torch.cuda.synchronize()
    for _ in range(5):
        assert all(torch.equal(a, c) for a, c in zip(step(), want))
    torch.cuda.synchronize()
    two = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [step(s.cuda_stream) for _ in range(4) for s in two]
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for out in outs for a, c in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want))
    _status_ok()


def test_offsets_past_32_bits():
    """P of more than 2^31 values."""
    M, F, K = 70000, 16384, 64
    X, W, b = _inputs(M, F, K, torch.bfloat16, 9)
    H, P = dga.gated_forward(X, W, b, save=True)
    rows = torch.tensor([0, 1, 32767, 32768, 65535, 65536, 65537, M - 1], device="cuda")
    want, eh, p, ep = ref.gated(X[rows], W, b, "silu")
    ref.within(H[rows], want, eh, "H")
    ref.within(P[rows], p, ep, "P")
    G = torch.randn(M, F, device="cuda", dtype=torch.bfloat16)
    dX, dW, db = dga.gated_backward(X, W, P, G, need_bias=True)
    want = ref.gated_grads(X[rows], W, P[rows], G[rows], "silu")
    ref.within(dX[rows], *want["dX"], "dX")
    cols = torch.tensor([0, 5, F - 1, F, F + 7, 2 * F - 1], device="cuda")
    gate = cols % F
    Ps = torch.cat([P[:, gate], P[:, F + gate]], 1)
    want = ref.gated_grads(X, torch.cat([W[gate], W[F + gate]]), Ps, G[:, gate].contiguous(), "silu")
    at = torch.arange(6, device="cuda") + 6 * (cols >= F)
    ref.within(dW[cols], want["dW"][0][at], want["dW"][1][at], "dW")
    ref.within(db[cols], want["db"][0][at], want["db"][1][at], "db")


def test_a_block_trained_as_it_is_used():
    """Up, gate, product and down projection, forward and backward, against fp64."""
    M, D, F = 200, 96, 160
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    X, W, Wd, T = r(M, D), r(2 * F, D) / 10, r(D, F) / 12, r(M, D)
    H, P = dga.gated_forward(X, W, save=True)
    Y = dga.linear_forward(H, Wd)
    G = Y - T
    dH, dWd, _ = dga.linear_backward(H, Wd, G, need_bias=False)
    dX, dW, _ = dga.gated_backward(X, W, P, dH)
    x, w, wd = (t.double().requires_grad_() for t in (X, W, Wd))
    p = x @ w.t()
    h = p[:, :F] / (1 + torch.exp(-p[:, :F])) * p[:, F:]
    ((h @ wd.t() - T.double()) ** 2).sum().div(2).backward()
    for got, want in ((dX, x.grad), (dW, w.grad), (dWd, wd.grad)):
        # three fp32 sums of up to 200 values behind one another, of mixed signs
        assert float((got.double() - want).norm() / want.norm()) < 3 * ref.sum_error(200)


# products with fewer tiles than the machine has places for, over a K that is cut: up to 128 rows and
# more, at sizes around the parts, with dX's K = 2F and dW's K = M in turn the long one
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,F,K", [(1, 520, 24), (3, 700, 40), (16, 2048, 130), (100, 2048, 300), (128, 1030, 515), (129, 512, 1000),
                                   (256, 4100, 260), (2050, 64, 96), (4096, 30, 130)])
def test_gradients_of_few_tiles(M, F, K, dtype):
    X, W, _ = _inputs(M, F, K, dtype, M + F)
    g = torch.Generator(device="cuda").manual_seed(M)
    P = (2 * torch.randn(M, 2 * F, device="cuda", generator=g)).to(dtype)
    G = torch.randn(M, F, device="cuda", generator=g).to(dtype)
    first = dga.gated_backward(X, W, P, G, activation="gelu_tanh", need_bias=True)
    want = ref.gated_grads(X, W, P, G, "gelu_tanh")
    for got, key in zip(first, ("dX", "dW", "db")):
        ref.within(got, *want[key], key)
    for _ in range(3):
        again = dga.gated_backward(X, W, P, G, activation="gelu_tanh", need_bias=True)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    _status_ok()


def test_gradients_with_the_least_workspace_and_one_too_small():
    M, F, K = 100, 1024, 256
    X, W, _ = _inputs(M, F, K, torch.bfloat16, 5)
    P, G = (torch.randn(M, n, device="cuda").bfloat16() for n in (2 * F, F))
    want = dga.gated_backward(X, W, P, G)
    need = dga.lib().dga_gated_backward_workspace_size(dga.BF16, M, F, K, K, K)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(dga.gated_backward(X, W, P, G, workspace=ws)[:2], want))
    with pytest.raises(dga.DgaError):
        dga.gated_backward(X, W, P, G, workspace=ws[:need - 256])
