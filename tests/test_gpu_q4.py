"""4-bit weights with group scales on the GPU against their definition in 64 bits
(tests/gated_reference.py)."""
import math

import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import gated_reference as ref

pytestmark = pytest.mark.gpu

HALVES = [torch.bfloat16, torch.float16]
OUT = {torch.float32: dga.F32, torch.bfloat16: dga.BF16, torch.float16: dga.F16}


def _weight(rows, cols, group, zeros, dtype, seed):
    """Random codes, scales of either sign's neighbourhood of 1/100, zero points over their range."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width, groups = (cols + 31) // 32 * 16, -(-cols // group)
    codes = torch.randint(0, 256, (rows, width), device="cuda", dtype=torch.uint8, generator=g)  # past cols too
    scales = (0.02 * torch.randn(rows, groups, device="cuda", generator=g)).to(dtype)
    z = torch.randint(0, 16, (rows, groups), device="cuda", dtype=torch.uint8, generator=g) if zeros else None
    return dga.Q4Tensor(cols, group, codes, scales, z)


def _values(Q):
    return ref.q4_values(Q.codes, Q.scales, Q.zeros, Q.cols, Q.group)


def _x(M, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, device="cuda", generator=g) * torch.exp(0.5 * torch.randn(K, device="cuda", generator=g))).to(dtype)


def _product(X, Q, bias=None):
    """(X W^T + bias, bound).  Many rows may go through the weight's values rounded to X's
    type, which adds half a step of each."""
    V = _values(Q)
    v, off = ref.product(X, V, bias)
    if X.shape[0] > 16:
        off = off + ref.HALF[X.dtype] * (X.double().abs() @ V.abs().t())
    return v, off


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, *HALVES])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 33), (2, 129), (40, 1000), (7, 256)])
def test_quantize_is_the_definition(rows, cols, dtype, zeros, group):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    W = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    W[:, cols // 2:] += 1.0
    if cols > 200:
        W[0] = 0.0
        W[1, 5], W[2, 40] = math.inf, math.nan
        W[3] = W[3].abs() + 1
        W[4] = -W[4].abs() - 1
        W[5] *= 1e-30 if dtype is not torch.float16 else 1e-7
    W = W.to(dtype)
    for st in HALVES:
        Q = dga.q4_quantize(W.cuda(), group, zeros, scale_dtype=st)
        q, s, z = ref.q4_quantize(W, group, zeros, st)
        fine = ~torch.isnan(s)
        assert torch.equal(torch.isnan(Q.scales.cpu()), ~fine)
        assert torch.equal(Q.scales.cpu()[fine], s[fine])
        at = fine.repeat_interleave(group, 1)[:, :cols]
        codes = Q.codes.cpu()
        assert torch.equal(ref.q4_unpack(codes, cols)[at], q[at])
        assert not ref.q4_unpack(codes, codes.shape[1] * 2)[:, cols:].any()
        if zeros:
            assert torch.equal(Q.zeros.cpu()[fine], z[fine])
        else:
            assert Q.zeros is None
        back = dga.q4_dequantize(Q).cpu().double()
        assert torch.equal(torch.isnan(back), ~at)
        # a value is off by half a scale s, by another half where the rounded zero point cuts
        # the range's end off, and by 15 times what rounding s took from the range: half a step
        # of s, or of the least number of its type
        sc = s.double().repeat_interleave(group, 1)[:, :cols].abs()
        assert bool(((back - W.double()).abs() <= (1 + 15 * ref.HALF[st]) * sc + 15 * ref.TINY[st])[at].all())


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("out", [torch.float32, *HALVES])
@pytest.mark.parametrize("rows,cols,group", [(1, 1, 32), (9, 70, 64), (33, 515, 128), (4, 512, 32)])
def test_dequantize_is_exact(rows, cols, group, out, dtype):
    for zeros in (False, True):
        Q = _weight(rows, cols, group, zeros, dtype, rows + cols)
        got = dga.q4_dequantize(Q, OUT[out])
        assert torch.equal(got, _values(Q).to(out))  # (q - z) s has at most 16 bits: fp64 to `out` rounds once


SIZES = [(1, 1, 1), (1, 16, 32), (1, 33, 31), (2, 100, 129), (4, 256, 1000), (7, 515, 512), (8, 64, 96), (9, 130, 520), (13, 300, 2048),
         (16, 1000, 264), (17, 48, 40), (31, 257, 300), (33, 200, 1030), (64, 130, 128), (65, 96, 515), (130, 333, 700), (300, 260, 256)]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K, group, dtype):
    for zeros, bias in ((False, True), (True, False)):
        Q = _weight(N, K, group, zeros, dtype, N + K)
        X = _x(M, K, dtype, M)
        b = torch.randn(N, device="cuda").to(dtype) if bias else None
        v, off = _product(X, Q, b)
        got = dga.q4_linear_forward(X, Q, b)
        assert got.dtype is dtype
        ref.within(got, v, off + ref.rounding(v, dtype) * (1 + 2.0 ** -7))
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,F,K", [(1, 1, 1), (1, 17, 64), (3, 100, 333), (5, 256, 1024), (8, 33, 40), (16, 515, 520), (20, 64, 128),
                                   (40, 130, 257), (100, 96, 512), (260, 150, 384)])
def test_gated(M, F, K, group, dtype):
    for i, name in enumerate(ref.ACTS):
        Q = _weight(2 * F, K, group, i % 2 == 0, dtype, F + K + i)
        X = _x(M, K, dtype, M + i)
        b = torch.randn(2 * F, device="cuda").to(dtype) if i % 3 else None
        P, off = _product(X, Q, b)
        H, eh = ref.gated_of(P, off, name, dtype)
        ref.within(dga.q4_gated_forward(X, Q, b, activation=name), H, eh, name)
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("M", [1, 5, 16, 40, 200])
def test_views_and_what_lies_around_the_results(M):
    """Rows further apart than their length, an X off 16 bytes, results inside larger
    arrays, NaN scales behind the last group and codes past the last column never read."""
    N, K, group, dtype = 70, 100, 32, torch.float16
    Q = _weight(N, K, group, True, dtype, 3)
    X = _x(M, K, dtype, 1)
    codes = torch.full((N, 96), 255, device="cuda", dtype=torch.uint8)
    codes[:, :64] = Q.codes
    scales = torch.full((N, 9), math.nan, device="cuda", dtype=dtype)
    scales[:, :4] = Q.scales
    zeros = torch.full((N, 7), 15, device="cuda", dtype=torch.uint8)
    zeros[:, :4] = Q.zeros + 16  # the upper half does not count
    Qv = dga.Q4Tensor(K, group, codes[:, :64], scales[:, :4], zeros[:, :4])
    b = torch.randn(N, device="cuda").to(dtype)
    v, off = _product(X, Q, b)
    H, eh = ref.gated_of(*_product(X, Q, b), "gelu", dtype)
    for shift, pad in ((0, 0), (0, 4), (1, 0), (3, 5), (8, 8)):
        xb = torch.full((M * (K + pad) + shift + 9,), math.nan, device="cuda", dtype=dtype)
        Xv = xb[shift:shift + M * (K + pad)].view(M, K + pad)[:, :K]
        Xv.copy_(X)
        for cols, call, want, bound in ((N, lambda y: dga.q4_linear_forward(Xv, Qv, b, Y=y), v, off + ref.rounding(v, dtype) * 1.01),
                                        (N // 2, lambda y: dga.q4_gated_forward(Xv, Qv, b, "gelu", H=y), H, eh)):
            yb = torch.full(((M + 1) * (cols + pad) + shift + 9,), 7.0, device="cuda", dtype=dtype)
            Y = yb[shift:shift + M * (cols + pad)].view(M, cols + pad)[:, :cols]
            assert call(Y) is Y
            ref.within(Y, want, bound)
            Y.fill_(7.0)
            assert bool((yb == 7.0).all())


@pytest.mark.parametrize("M", [1, 3, 12, 40, 200])
def test_infinities_stay_in_their_rows_and_columns(M):
    """An infinity or NaN in a token, or a NaN scale, reaches that token's outputs, or that
    row's, and nothing else."""
    N, K, dtype = 80, 300, torch.bfloat16
    Q = _weight(N, K, 64, True, dtype, 4)
    X = _x(M, K, dtype, 2)
    want = dga.q4_linear_forward(X, Q)
    Xb = X.clone()
    Xb[M // 2, 17], Xb[M // 2, 290] = math.inf, math.nan
    got = dga.q4_linear_forward(Xb, Q)
    keep = torch.arange(M, device="cuda") != M // 2
    assert bool(torch.isnan(got[M // 2]).all()) and torch.equal(got[keep], want[keep])
    Q.scales[11, 2] = math.nan
    got = dga.q4_linear_forward(X, Q)
    keep = torch.arange(N, device="cuda") != 11
    assert bool(torch.isnan(got[:, 11]).all()) and torch.equal(got[:, keep], want[:, keep])


def test_empty_sizes():
    for dtype in HALVES:
        Q = _weight(6, 40, 32, True, dtype, 1)
        assert dga.q4_linear_forward(torch.zeros(0, 40, device="cuda", dtype=dtype), Q).shape == (0, 6)
        assert dga.q4_gated_forward(torch.zeros(0, 40, device="cuda", dtype=dtype), Q).shape == (0, 3)
        E = dga.Q4Tensor(0, 32, torch.zeros(6, 0, device="cuda", dtype=torch.uint8), torch.zeros(6, 0, device="cuda", dtype=dtype))
        b = torch.arange(6, device="cuda").to(dtype) + 1
        X = torch.zeros(4, 0, device="cuda", dtype=dtype)
        assert torch.equal(dga.q4_linear_forward(X, E, b), b.expand(4, 6))
        assert torch.equal(dga.q4_gated_forward(X, E, b, "relu"), (b[:3] * b[3:]).expand(4, 3))
        assert dga.q4_dequantize(E).shape == (6, 0)


@pytest.mark.parametrize("M", [1, 13, 40, 200])
def test_graph_streams_and_repeats(M):
    dtype = torch.bfloat16
    Q = _weight(512, 640, 128, True, dtype, 6)
    X = _x(M, 640, dtype, 7)

    def step(stream=None):
        return dga.q4_linear_forward(X, Q, stream=stream), dga.q4_gated_forward(X, Q, activation="silu", stream=stream)

    want = step()
    torch.cuda.synchronize()
    two = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [step(s.cuda_stream) for _ in range(4) for s in two]
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for out in outs for a, c in zip(out, want))
    graphs = []
    for _ in range(2):  # two graphs, replayed at once
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        graphs.append((graph, got))
    for _ in range(3):
        for (graph, got), s in zip(graphs, two):
            with torch.cuda.stream(s):
                for t in got:
                    t.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for _, got in graphs for a, c in zip(got, want))
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


def test_offsets_past_32_bits():
    """Codes and results past 2^31 bytes and values."""
    N, K, dtype = 1 << 20, 4160, torch.bfloat16
    Q = _weight(N, K, 128, True, dtype, 8)
    assert Q.codes.numel() > 1 << 31
    rows = torch.tensor([0, 5, 500000, 1000000, N // 2 - 1, N // 2, N - 1], device="cuda")
    S = dga.Q4Tensor(K, 128, Q.codes[rows], Q.scales[rows], Q.zeros[rows])
    X = _x(3, K, dtype, 9)
    v, off = _product(X, S)
    ref.within(dga.q4_linear_forward(X, Q)[:, rows], v, off + ref.rounding(v, dtype) * 1.01)
    at = torch.tensor([0, 77, N // 2 - 1], device="cuda")
    G = dga.Q4Tensor(K, 128, *(torch.cat([t[at], t[at + N // 2]]) for t in (Q.codes, Q.scales, Q.zeros)))
    H, eh = ref.gated_of(*_product(X, G), "silu", dtype)
    ref.within(dga.q4_gated_forward(X, Q)[:, at], H, eh)
    Q = _weight(70000, 160, 32, False, dtype, 10)
    X = _x(31000, 160, dtype, 11)  # 2.2e9 results
    Y = dga.q4_linear_forward(X, Q)
    at = torch.tensor([0, 3, 30719, 30720, 30999], device="cuda")
    v, off = ref.product(X[at], _values(Q))
    off = off + ref.HALF[dtype] * (X[at].double().abs() @ _values(Q).abs().t())
    ref.within(Y[at], v, off + ref.rounding(v, dtype) * 1.01)


def test_a_block_quantised_and_served():
    """A trained block's weights to 4 bits; one token and a prompt through it."""
    D, F, dtype = 256, 384, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(2)
    W = (torch.randn(2 * F, D, device="cuda", generator=g) / 16).to(dtype)
    Wd = (torch.randn(D, F, device="cuda", generator=g) / 20).to(dtype)
    Q, Qd = dga.q4_quantize(W, 64), dga.q4_quantize(Wd, 128, zeros=False)
    for M in (1, 9, 150):
        X = _x(M, D, dtype, M)
        Y = dga.q4_linear_forward(dga.q4_gated_forward(X, Q), Qd)
        P, off = _product(X, Q)
        H, eh = ref.gated_of(P, off, "silu", dtype)
        V = _values(Qd)
        v = H @ V.t()
        bound = eh @ V.abs().t() + (ref.sum_error(F) + ref.HALF[dtype]) * ((H.abs() + eh) @ V.abs().t())
        ref.within(Y, v, bound + ref.rounding(v, dtype) * 1.01)
        # the same block before it was quantised: its gated layer on the values that the codes stand for
        same = dga.gated_forward(X, dga.q4_dequantize(Q, dga.BF16))
        assert float((same.double() - H).norm() / H.norm()) < 4 * ref.HALF[dtype]


# rows of X around the tensor-core kernel's stages (128, 208, 256 to a tile), K cut among the CTAs of a
# cluster unevenly, a weight small and large enough for either kernel at 33 to 64 rows
@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(33, 2050, 2090), (64, 600, 7000), (65, 129, 4100), (130, 257, 1290), (207, 384, 1000), (209, 128, 2049),
                                   (256, 300, 8200), (257, 120, 770), (600, 260, 2111), (1024, 64, 513), (1025, 130, 260)])
def test_linear_on_the_tensor_cores(M, N, K, group, dtype):
    Q = _weight(N, K, group, M % 2 == 0, dtype, N + K)
    X = _x(M, K, dtype, M)
    b = torch.randn(N, device="cuda").to(dtype) if M % 2 else None
    v, off = _product(X, Q, b)
    got = dga.q4_linear_forward(X, Q, b)
    ref.within(got, v, off + ref.rounding(v, dtype) * (1 + 2.0 ** -7))
    for _ in range(3):
        assert torch.equal(dga.q4_linear_forward(X, Q, b), got)
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,F,K", [(33, 1100, 2090), (64, 130, 5000), (65, 70, 2100), (128, 129, 1030), (129, 200, 515), (400, 64, 3000),
                                   (512, 131, 256), (513, 96, 1000), (700, 130, 515)])
def test_gated_on_the_tensor_cores(M, F, K, group, dtype):
    name = ref.ACTS[(M + F) % 5]
    Q = _weight(2 * F, K, group, M % 2 == 1, dtype, F + K)
    X = _x(M, K, dtype, M)
    b = torch.randn(2 * F, device="cuda").to(dtype) if M % 2 else None
    P, off = _product(X, Q, b)
    H, eh = ref.gated_of(P, off, name, dtype)
    got = dga.q4_gated_forward(X, Q, b, activation=name)
    ref.within(got, H, eh, name)
    assert torch.equal(dga.q4_gated_forward(X, Q, b, activation=name), got)
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("M", [48, 256, 300])
@pytest.mark.parametrize("group", [32, 128])
def test_tensor_core_launches_beside_one_another(M, group):
    """Long loops of few stages on two streams at once, whose warps run apart from one another."""
    dtype = torch.float16
    Q = [_weight(1200, 8192, group, i == 0, dtype, i) for i in range(2)]
    X = _x(M, 8192, dtype, M)
    want = [(dga.q4_linear_forward(X, q), dga.q4_gated_forward(X, q)) for q in Q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Q]
    for _ in range(20):
        got = [(dga.q4_linear_forward(X, q, stream=s.cuda_stream), dga.q4_gated_forward(X, q, stream=s.cuda_stream)) for q, s in zip(Q, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


def test_infinite_scales_stay_what_they_are():
    """K that ends inside a block of columns: (q - z) inf times X, and no NaN from what lies past K."""
    for dtype in HALVES:
        for M in (4, 70, 300):
            Q = _weight(130, 100, 64, False, dtype, 1)
            Q.codes.fill_(0x99)  # q - 8 = 1
            Q.scales.fill_(1.0)
            Q.scales[5, 1] = math.inf
            X = torch.ones(M, 100, device="cuda", dtype=dtype)
            Y = dga.q4_linear_forward(X, Q)
            want = torch.full_like(Y, 100.0)
            want[:, 5] = math.inf
            assert torch.equal(Y, want)
