"""4-bit microscaled quantisation, its inverse and its products on the GPU,
against the formats' definition in fp64 (tests/mx_reference.py)."""
import numpy as np
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
import oracle
from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

FMT = [dga.MXFP4, dga.NVFP4]
TYPES = [torch.float32, torch.bfloat16, torch.float16]
OUT = {torch.float32: dga.F32, torch.bfloat16: dga.BF16, torch.float16: dga.F16}


def _values(rows, cols, seed, dtype=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, cols // 7 + 1, generator=g)).repeat_interleave(7, 1)[:, :cols]
    return x.to(dtype)


def _np(t):
    return t.double().numpy()


def _factor(x, fmt):
    """A power-of-two tensor scale for NVFP4 (scaling by it is exact)."""
    if fmt == dga.MXFP4:
        return None, 1.0
    f = float(2.0 ** np.ceil(np.log2(float(x.abs().max()) / 2688.0)))
    return torch.tensor([f], device="cuda"), f


def _parts(q):
    """(codes, scale bytes) of an MXTensor on the host."""
    return (ref.unpack_codes(q.codes.cpu().numpy(), q.cols),
            ref.untile_scales(q.scales.cpu().numpy(), q.rows, q.cols, q.format))


def _sync_ok():
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 15), (3, 16), (5, 33), (130, 257), (31, 1000), (257, 129), (64, 512)])
def test_codes_and_scales_are_the_definitions(fmt, dtype, transpose, rows, cols):
    x = _values(rows, cols, rows * 1000 + cols, dtype)
    f, fv = _factor(x, fmt)
    q = dga.mx_quantize(x.cuda(), fmt, transpose=transpose, tensor_scale=f)
    want_c, want_s = ref.quantize(_np(x).T if transpose else _np(x), fmt, fv)
    got_c, got_s = _parts(q)
    assert q.shape == want_c.shape
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    # the codes between K and the row's end are zero, so that products may read them
    full = ref.unpack_codes(q.codes.cpu().numpy(), q.codes.shape[1] * 2)
    assert not full[:, q.cols:].any()
    for out in TYPES:
        y = dga.mx_dequantize(q, OUT[out]).cpu()
        want = torch.from_numpy(ref.dequantize(want_c, want_s, fmt, fv)).float().to(out)
        assert torch.equal(y, want)


def test_every_bf16_value_and_tie():
    """All finite bf16 magnitudes as one block's second value beside a fixed
    largest one: every rounding tie of the two formats is among them."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    for fmt in FMT:
        b = ref.BLOCK[fmt]
        x = torch.zeros(v.numel(), 2 * b, dtype=torch.bfloat16)
        x[:, 0], x[:, b] = v, 5.0  # alone in its block; beside a 5
        x[:, b + 1] = -torch.minimum(v, torch.tensor(5.0, dtype=torch.bfloat16))
        q = dga.mx_quantize(x.cuda(), fmt)
        want_c, want_s = ref.quantize(_np(x), fmt)
        got_c, got_s = _parts(q)
        assert np.array_equal(got_s, want_s), fmt
        assert np.array_equal(got_c, want_c), fmt


@pytest.mark.parametrize("fmt", FMT)
def test_extremes(fmt):
    """Zero blocks, subnormals, the largest values, infinities and NaN."""
    b = ref.BLOCK[fmt]
    x = torch.zeros(1, 8 * b)
    x[0, b] = 1e-45
    x[0, 2 * b:3 * b] = torch.linspace(-1e-38, 1e-38, b)
    x[0, 3 * b] = 3.4e38
    x[0, 3 * b + 1] = -2.9e38
    x[0, 4 * b + 3] = float("inf")
    x[0, 5 * b + 7] = float("nan")
    x[0, 5 * b + 8] = 1.0
    x[0, 6 * b:7 * b] = 448 * 6 * 4.0  # past E4M3's largest scale
    x[0, 7 * b:] = -0.0
    q = dga.mx_quantize(x.cuda(), fmt)
    want_c, want_s = ref.quantize(_np(x), fmt)
    got_c, got_s = _parts(q)
    assert np.array_equal(got_s, want_s)
    finite = np.isfinite(np.repeat(np.where((want_s == (0xFF if fmt == dga.MXFP4 else 0x7F)), np.nan, 1.0), b, axis=1))
    assert np.array_equal(got_c[finite], want_c[finite])
    y = dga.mx_dequantize(q).cpu().numpy()
    assert np.isnan(y[0, 4 * b:6 * b]).all() and np.isfinite(np.delete(y[0], range(4 * b, 6 * b))).all()


def test_general_tensor_scale():
    """A factor that is no power of two: the roundings are fp32's, so a value
    may fall to the other side of a tie, and no further."""
    x = _values(64, 640, 5)
    f = float(x.abs().max()) / 2688.0
    q = dga.mx_quantize(x.cuda(), dga.NVFP4, tensor_scale=torch.tensor([f], device="cuda"))
    want = ref.dequantize(*ref.quantize(_np(x), dga.NVFP4, f), dga.NVFP4, f)
    got = dga.mx_dequantize(q).cpu().double().numpy()
    off = np.abs(got - want) > 1e-6 * np.abs(want)
    assert off.mean() < 1e-4
    for tiny in (1e-30, 1e-38, 1e30):  # units past where the quotient is corrected
        t = torch.tensor([tiny], device="cuda")
        xs = (x * tiny).cuda()
        y = dga.mx_dequantize(dga.mx_quantize(xs, dga.NVFP4, tensor_scale=t)).cpu().double().numpy()
        w = ref.dequantize(*ref.quantize(_np(xs.cpu()), dga.NVFP4, tiny), dga.NVFP4, tiny)
        assert (np.abs(y - w) > 1e-6 * np.abs(w) + 1e-44).mean() < 1e-4


def test_strided_and_column_major_inputs():
    base = _values(70, 300, 9).cuda()
    for fmt in FMT:
        for view in (base[:, 3:200], base[5:60, 1:], base.t(), base[::2, :], base.t()[7:, 2:]):
            q = dga.mx_quantize(view, fmt)
            want_c, want_s = ref.quantize(_np(view.cpu()), fmt)
            got_c, got_s = _parts(q)
            assert np.array_equal(got_c, want_c) and np.array_equal(got_s, want_s)
            t = dga.mx_quantize(view, fmt, transpose=True)
            want_c, want_s = ref.quantize(_np(view.cpu()).T, fmt)
            got_c, got_s = _parts(t)
            assert np.array_equal(got_c, want_c) and np.array_equal(got_s, want_s)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,ld", [(1, 70, 70), (3, 5, 7), (9, 95, 95), (33, 257, 259), (5, 1030, 1037)])
@pytest.mark.parametrize("offset", range(8))
def test_rows_at_any_alignment(fmt, dtype, rows, cols, ld, offset):
    """Sources and results whose rows start on any element, at the ends of their
    memory, between neighbours that must not be taken in or changed."""
    x = _values(rows, cols, 7 * rows + cols + offset, dtype)
    f, fv = _factor(x, fmt)
    memory = torch.full((offset + (rows - 1) * ld + cols,), 3e4, dtype=dtype, device="cuda")
    X = memory.as_strided((rows, cols), (ld, 1), offset)
    X.copy_(x)
    q = dga.mx_quantize(X, fmt, tensor_scale=f)
    want_c, want_s = ref.quantize(_np(x), fmt, fv)
    got_c, got_s = _parts(q)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    plain = dga.mx_dequantize(q, out_dtype=OUT[dtype])
    memory.fill_(5.0)
    st = dga.dga_mx_dequantize(fmt, OUT[dtype], rows, cols, q.codes.data_ptr(), q.codes.stride(0), q.scales.data_ptr(),
                               f.data_ptr() if f is not None else None, X.data_ptr(), ld, torch.cuda.current_stream().cuda_stream)
    assert st == dga.OK
    assert torch.equal(X, plain)
    assert torch.equal(X.cpu(), torch.from_numpy(ref.dequantize(want_c, want_s, fmt, fv)).to(dtype))
    X.fill_(5.0)
    assert bool((memory == 5.0).all())


def _pair(M, N, K, fmt, seed=0):
    a, b = _values(M, K, seed + 1), _values(N, K, seed + 2)
    fa, va = _factor(a, fmt)
    fb, vb = _factor(b, fmt)
    qa, qb = dga.mx_quantize(a.cuda(), fmt, tensor_scale=fa), dga.mx_quantize(b.cuda(), fmt, tensor_scale=fb)
    A = ref.dequantize(*ref.quantize(_np(a), fmt, va), fmt, va)
    B = ref.dequantize(*ref.quantize(_np(b), fmt, vb), fmt, vb)
    return qa, qb, A, B


def _ulp(x, dtype):
    if dtype == torch.float32:
        return np.abs(x) * 2.0 ** -23
    return oracle.ulp_bf16(x) if dtype == torch.bfloat16 else oracle.ulp_f16(x)


SHAPES = [(1, 1, 1), (1, 128, 64), (2, 127, 100), (5, 129, 255), (16, 300, 256), (17, 300, 257), (33, 500, 1000),
          (64, 1000, 1111), (65, 64, 2000), (100, 700, 4096), (129, 257, 513), (200, 640, 3000), (255, 100, 64),
          (256, 256, 256), (257, 255, 300), (300, 1, 77), (511, 700, 1025), (700, 513, 2049)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(fmt, M, N, K):
    qa, qb, A, B = _pair(M, N, K, fmt)
    want, bound = A @ B.T, ref.product_bound(A, B, K)
    for dtype in TYPES:
        got = dga.mx_gemm(qa, qb, out_dtype=OUT[dtype]).cpu().double().numpy()
        _sync_ok()
        if dtype == torch.float16:
            keep = np.abs(want) < 60000
        else:
            keep = np.ones_like(want, bool)
        err = np.abs(got - want)
        tol = bound + _ulp(want, dtype)
        assert (err <= tol)[keep].all(), (dtype, float((err / np.maximum(tol, 1e-300))[keep].max()))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M,N,K", [(3, 140, 520), (40, 257, 700), (150, 260, 800), (300, 520, 600)])
def test_integers_are_exact_and_alpha_beta_bias(fmt, M, N, K):
    """Small integers with unit scales: every sum is exact, so that the output is
    alpha * sum + beta * C + bias to the last bit, in C's own strides."""
    g = torch.Generator().manual_seed(M)
    lev = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0, -1.0, -2.0, -4.0, -6.0])
    a, b = (lev[torch.randint(0, 10, (r, K), generator=g)] for r in (M, N))
    a[:, ::16] = 6.0  # every block's largest value is 6: unit scales
    b[:, ::16] = 6.0
    qa, qb = dga.mx_quantize(a.cuda(), fmt), dga.mx_quantize(b.cuda(), fmt)
    base = torch.randint(-50, 50, (M, N + 3), generator=g).float().cuda()
    bias = torch.randint(-9, 9, (N,), generator=g).float().cuda()
    s = a.double() @ b.double().T
    C = base[:, 1:N + 1]
    want = 2.0 * s - 0.5 * C.cpu().double() + bias.cpu().double()
    keep = base.clone()
    dga.mx_gemm(qa, qb, C, alpha=2.0, beta=-0.5, bias=bias)
    _sync_ok()
    assert torch.equal(C.cpu().double(), want)
    assert torch.equal(base[:, 0], keep[:, 0]) and torch.equal(base[:, N + 1:], keep[:, N + 1:])
    # beta == 0 does not read C; alpha == 0 does not read the operands
    C2 = torch.full((M, N), float("nan"), device="cuda")
    assert torch.equal(dga.mx_gemm(qa, qb, C2).cpu().double(), s)
    C3 = torch.ones((M, N), device="cuda")
    assert torch.equal(dga.mx_gemm(qa, qb, C3, alpha=0.0, beta=3.0, bias=bias).cpu(), (3.0 + bias.cpu()).expand(M, N))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("M", [1, 20, 120, 300])
def test_nan_blocks_stay_in_their_rows(fmt, M):
    """A NaN in one row of A and one of B spoils that row and column of C only;
    what lies past the matrices in memory spoils nothing."""
    N, K = 200, 330
    a, b = _values(M, K, 1), _values(N, K, 2)
    a[M // 2, 100], b[77, 329] = float("nan"), float("inf")
    C = dga.mx_gemm(dga.mx_quantize(a.cuda(), fmt), dga.mx_quantize(b.cuda(), fmt), out_dtype=dga.F32).cpu()
    _sync_ok()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[M // 2], bad[:, 77] = True, True
    assert torch.equal(torch.isnan(C), bad)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (1, 1000, 2048), (7, 513, 1111), (16, 300, 5000), (17, 300, 800), (90, 300, 700),
                                   (400, 300, 520)])
def test_linear_forward(fmt, dtype, T, N, K):
    """The layer equals quantisation and product called apart, bit for bit."""
    x, w = _values(T, K, 3, dtype), _values(N, K, 4) / K ** 0.5
    f, _ = _factor(x, fmt)
    W = dga.mx_quantize(w.cuda(), fmt)
    bias = torch.randn(N, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    y = dga.mx_linear_forward(x.cuda(), W, bias, tensor_scale=f)
    z = dga.mx_gemm(dga.mx_quantize(x.cuda(), fmt, tensor_scale=f), W, out_dtype=OUT[dtype], bias=bias)
    _sync_ok()
    assert y.dtype == dtype and torch.equal(y, z)
    assert torch.equal(y, dga.mx_linear_forward(x.cuda(), W, bias, tensor_scale=f))  # repeats bit for bit


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T,N,K", [(33, 40, 50), (300, 257, 129)])
def test_linear_backward(fmt, T, N, K):
    """dX and dW are the products of the rounded operands."""
    x, w, g = _values(T, K, 5), _values(N, K, 6), _values(T, N, 7)
    dX, dW, db = dga.mx_linear_backward(x.cuda(), w.cuda(), g.cuda(), fmt)
    _sync_ok()

    def near(t):
        return ref.dequantize(*ref.quantize(t, fmt), fmt)
    X, W, G = _np(x), _np(w), _np(g)
    for got, A, B, n in ((dX, near(G), near(W.T), N), (dW, near(G.T), near(X.T), T)):
        want = A @ B.T
        tol = ref.product_bound(A, B, n) + _ulp(want, torch.float32)
        assert (np.abs(got.cpu().double().numpy() - want) <= tol).all()
    assert np.allclose(db.cpu().double().numpy(), G.sum(0), rtol=1e-5, atol=1e-4)


def test_on_another_stream_and_in_a_graph():
    x, w = _values(9, 1000, 1).cuda(), _values(600, 1000, 2).cuda()
    W = dga.mx_quantize(w)
    want = dga.mx_linear_forward(x, W)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = dga.mx_linear_forward(x, W)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    xin = x.clone()
    with torch.cuda.graph(graph):
        out = dga.mx_linear_forward(xin, W)
    xin.copy_(x * 2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dga.mx_linear_forward(x * 2, W))


def test_a_given_stream_owns_what_is_allocated():
    """Memory freed while the current stream has yet to read it is not handed
    out to a call on another stream."""
    x = _values(256, 1024, 3).cuda()
    q = dga.mx_quantize(x)
    want = dga.mx_dequantize(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in (lambda: dga.mx_dequantize(q, stream=s.cuda_stream), lambda: dga.orthogonalize(x, stream=s.cuda_stream),
                 lambda: dga.mx_gemm(q, q, out_dtype=dga.F32, stream=s.cuda_stream)):
        old = torch.full_like(want, 7.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        copy = old.clone()
        del old
        call()
        torch.cuda.synchronize()
        assert bool((copy == 7.0).all())
    assert torch.equal(dga.mx_dequantize(q, stream=torch.cuda.default_stream().cuda_stream), want)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtypes", [(torch.bfloat16,) * 3, (torch.float32, torch.bfloat16, torch.float16)])
@pytest.mark.parametrize("T,N,K", [(1, 1, 1), (5, 130, 67), (33, 40, 50), (300, 257, 129), (64, 520, 300)])
def test_linear_backward_is_its_parts(fmt, dtypes, T, N, K):
    """One call equals quantisations, products and sum called apart, bit for bit,
    for row-major operands, views and column-major ones."""
    base = [_values(T, K + 3, 5, dtypes[0]).cuda(), _values(N, K + 3, 6, dtypes[1]).cuda(), _values(T, N + 3, 7, dtypes[2]).cuda()]
    x, w, g = (t[:, 1:-2] for t in base)
    f = [_factor(t.cpu(), fmt)[0] for t in (x, w, g)]
    want_dX = dga.mx_gemm(dga.mx_quantize(g, fmt, tensor_scale=f[2]), dga.mx_quantize(w, fmt, True, f[1]), out_dtype=OUT[dtypes[2]])
    want_dW = dga.mx_gemm(dga.mx_quantize(g, fmt, True, f[2]), dga.mx_quantize(x, fmt, True, f[0]), out_dtype=OUT[dtypes[2]])
    for a, b, c in ((x, w, g), (x.contiguous(), w.contiguous(), g.contiguous()), (x.t().contiguous().t(), w, g)):
        dX, dW, db = dga.mx_linear_backward(a, b, c, fmt, tensor_scales=tuple(f))
        _sync_ok()
        assert torch.equal(dX, want_dX) and torch.equal(dW, want_dW) and torch.equal(db, dga.sum_rows(g))
    assert dga.mx_linear_backward(x, w, g, fmt, need_bias=False)[2] is None


def test_linear_backward_of_nothing():
    for T, N, K in ((0, 5, 7), (4, 0, 7), (4, 5, 0)):
        x, w, g = torch.ones(T, K, device="cuda"), torch.ones(N, K, device="cuda"), torch.ones(T, N, device="cuda")
        dX, dW, db = dga.mx_linear_backward(x, w, g)
        _sync_ok()
        assert dX.shape == (T, K) and not dX.any()
        assert dW.shape == (N, K) and not dW.any()
        assert torch.equal(db, torch.full((N,), float(T), device="cuda"))


@pytest.mark.parametrize("fmt", FMT)
def test_offsets_past_32_bits(fmt):
    """Sources, values and products of more than 2^31 elements: their last rows
    and columns are those of the same rows alone."""
    rows, cols = 65536 + 128, 33000
    X = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    for r in range(0, rows, 8208):
        X[r:r + 8208] = torch.randn(8208, cols, device="cuda", generator=g)
    tail = X[-128:].contiguous()
    q, alone = dga.mx_quantize(X, fmt), dga.mx_quantize(tail, fmt)
    assert torch.equal(q.codes[-128:], alone.codes)
    per = alone.scales.numel()
    assert torch.equal(q.scales.flatten()[-per:], alone.scales.flatten())
    assert torch.equal(dga.mx_dequantize(q, out_dtype=dga.BF16)[-128:], dga.mx_dequantize(alone, out_dtype=dga.BF16))
    t = dga.mx_quantize(X, fmt, transpose=True)
    t_alone = dga.mx_quantize(X[:, -104:].contiguous(), fmt, transpose=True)
    assert torch.equal(t.codes[-104:], t_alone.codes)
    del X, q, t
    # one-hot rows: C's last rows and columns are entries of A and B
    M, N, K = 66000, 33000, 64
    A = torch.zeros(M, K, device="cuda")
    A[torch.arange(M, device="cuda"), torch.arange(M, device="cuda") % K] = 6.0
    B = torch.randint(-3, 4, (N, K), device="cuda", generator=g).float()
    B[:, ::16] = 6.0  # every block's largest, so that the scales are exact
    C = dga.mx_gemm(dga.mx_quantize(A, fmt), dga.mx_quantize(B, fmt), out_dtype=dga.BF16)
    _sync_ok()
    for r in (0, M - 300):
        want = B[:, (torch.arange(r, r + 300, device="cuda") % K)].mT
        assert torch.equal(C[r:r + 300].float(), 6.0 * want)


def test_empty():
    e = torch.empty(0, 40, device="cuda")
    q = dga.mx_quantize(e)
    assert q.shape == (0, 40) and dga.mx_dequantize(q).shape == (0, 40)
    w = dga.mx_quantize(torch.ones(5, 40, device="cuda"))
    assert dga.mx_gemm(q, w).shape == (0, 5)
    assert dga.mx_linear_forward(e, w).shape == (0, 5)
    k0 = dga.mx_quantize(torch.empty(3, 0, device="cuda"))
    k1 = dga.mx_quantize(torch.empty(4, 0, device="cuda"))
    bias = torch.arange(4, device="cuda", dtype=torch.float32)
    assert torch.equal(dga.mx_gemm(k0, k1, out_dtype=dga.F32, bias=bias), bias.expand(3, 4))


def test_refusals():
    x = torch.ones(4, 64, device="cuda")
    q, n = dga.mx_quantize(x), dga.mx_quantize(x, dga.NVFP4)
    f = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        dga.mx_quantize(x, dga.MXFP4, tensor_scale=f)
    with pytest.raises(ValueError):
        dga.mx_quantize(x, dga.NVFP4, tensor_scale=f.double())
    with pytest.raises(TypeError):
        dga.mx_quantize(x.to(torch.int8))
    with pytest.raises(ValueError):
        dga.mx_quantize(x.reshape(2, 2, 64))
    with pytest.raises(ValueError):
        dga.mx_quantize(x.cpu())
    with pytest.raises(TypeError):
        dga.mx_gemm(q, n)
    with pytest.raises(ValueError):
        dga.mx_gemm(q, dga.mx_quantize(torch.ones(4, 65, device="cuda")))
    with pytest.raises(ValueError):
        dga.mx_gemm(q, q, beta=1.0)
    with pytest.raises(ValueError):
        dga.mx_gemm(q, q, torch.empty(4, 5, device="cuda"))
    with pytest.raises(ValueError):
        dga.mx_gemm(q, q, bias=torch.ones(4, device="cuda"))  # not the output's type
    with pytest.raises(ValueError):
        dga.mx_linear_forward(torch.ones(2, 63, device="cuda"), q)
    with pytest.raises(dga.DgaError):
        dga.mx_linear_forward(torch.ones(17, 64, device="cuda"), q,
                              workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
