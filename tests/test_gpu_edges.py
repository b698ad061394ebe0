"""Edges of the 4-bit and orthogonalisation calls on the GPU: zero tensors,
values far past a tensor's factor, host threads, devices and eps = 0."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import dense_gemm_accelerator_gb300 as dga
from tests import mx_reference as ref

pytestmark = pytest.mark.gpu

FMT = [dga.MXFP4, dga.NVFP4]
TYPES = [torch.float32, torch.bfloat16, torch.float16]
OUT = {torch.float32: dga.F32, torch.bfloat16: dga.BF16, torch.float16: dga.F16}


def _parts(q):
    """(codes, scale bytes) of an MXTensor on the host."""
    return (ref.unpack_codes(q.codes.cpu().numpy(), q.cols),
            ref.untile_scales(q.scales.cpu().numpy(), q.rows, q.cols, q.format))


def _sync_ok():
    assert dga.dga_sync_status(torch.cuda.current_stream().cuda_stream) == dga.OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 13, 40, 300])
def test_a_zero_tensor_with_its_zero_factor(dtype, rows):
    """max|X| / 2688 of a zero tensor is 0: its blocks are zeros still."""
    N, K = 130, 200
    zero = torch.zeros(1, device="cuda")
    X = torch.zeros(rows, K, dtype=dtype, device="cuda")
    X[0, 3] = -0.0
    for transpose in (False, True):
        q = dga.mx_quantize(X, dga.NVFP4, transpose=transpose, tensor_scale=zero)
        codes, scales = _parts(q)
        assert not scales.any() and not (codes & 7).any()
        assert not dga.mx_dequantize(q).any()
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(1)).cuda()
    W = dga.mx_quantize(w, dga.NVFP4)
    bias = torch.arange(N, device="cuda").to(dtype)
    assert torch.equal(dga.mx_linear_forward(X, W, bias, tensor_scale=zero), bias.expand(rows, N))
    G = torch.randn(rows, N, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    dX, dW, db = dga.mx_linear_backward(X, w, G, dga.NVFP4, tensor_scales=(zero, None, None))
    assert not dW.any() and bool(torch.isfinite(dX).all())
    dX, dW, db = dga.mx_linear_backward(X, w, torch.zeros_like(G), dga.NVFP4, tensor_scales=(zero, None, zero))
    _sync_ok()
    assert not dX.any() and not dW.any() and not db.any()


def test_zero_blocks_beside_others_keep_a_zero_scale():
    X = torch.zeros(4, 64, device="cuda")
    X[1, 16:32] = 3.0
    for f in (None, torch.full((1,), 2.0 ** -120, device="cuda"), torch.full((1,), 2.0 ** 120, device="cuda")):
        _, scales = _parts(dga.mx_quantize(X, dga.NVFP4, tensor_scale=f))
        want = np.zeros((4, 4), np.uint8)
        want[1, 1] = ref.quantize(X.cpu().double().numpy(), dga.NVFP4, 1.0 if f is None else float(f))[1][1, 1]
        assert np.array_equal(scales, want)


@pytest.mark.parametrize("rows", [9, 40])
@pytest.mark.parametrize("log2f", [-14, -40, -80, -88, -120, 30, 80, 100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_far_past_a_tensors_factor(dtype, log2f, rows):
    """Quotients over fp32's range are the largest codes, of the values' signs,
    and the largest scales; as far below it they are zeros."""
    K = 16 * 24
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K, generator=g)
    exponents = torch.randint(-120, 124, (rows, K // 16), generator=g).float()
    exponents[:, ::3] = torch.randint(90, 124, (rows, K // 48), generator=g).float()
    x = (x.reshape(rows, -1, 16) * torch.exp2(exponents)[..., None]).reshape(rows, K).clamp(-3.3e38, 3.3e38)
    x[0, 0], x[0, 1], x[0, 2] = -2e37, 2e37, -1e3
    x = x.to(dtype)
    factor = torch.tensor([2.0 ** log2f], device="cuda")
    want_c, want_s = ref.quantize(x.double().numpy(), dga.NVFP4, 2.0 ** log2f)
    for q in (dga.mx_quantize(x.cuda(), dga.NVFP4, tensor_scale=factor),
              dga.mx_quantize(x.t().contiguous().cuda(), dga.NVFP4, transpose=True, tensor_scale=factor)):
        codes, scales = _parts(q)
        assert np.array_equal(scales, want_s)
        # a zero unit gives zeros, whatever their sign
        live = np.repeat(want_s != 0, 16, axis=1) | ((codes & 7) != 0)
        assert np.array_equal(codes[live], want_c[live])


@pytest.mark.parametrize("rows", [3, 20])
def test_the_layer_on_values_far_past_the_factor(rows):
    """The same codes where the product quantises (up to 16 rows) and where it does not."""
    x = torch.zeros(rows, 64, device="cuda")
    x[:, 5], x[:, 20] = -2e37, 3e38
    f = torch.tensor([1e-4], device="cuda")
    w = torch.zeros(8, 64, device="cuda")
    w[0, 5] = w[1, 20] = 6.0
    y = dga.mx_linear_forward(x, dga.mx_quantize(w, dga.NVFP4), tensor_scale=f)
    _sync_ok()
    unit = float(np.float32(448) * np.float32(1e-4))
    want = torch.zeros(rows, 8)
    want[:, 0], want[:, 1] = -36.0 * unit, 36.0 * unit
    assert torch.allclose(y.cpu(), want, rtol=1e-6, atol=0)


def test_host_threads_with_updates_of_other_sizes():
    """Sizes that take different amounts of shared memory of one kernel, called
    at the same time by several threads."""
    g = torch.Generator().manual_seed(4)
    inputs = [torch.randn(64, 64, generator=g).cuda(), torch.randn(100, 30, 190, generator=g).cuda()]
    torch.cuda.synchronize()
    codes, start = [], threading.Barrier(4)
    coefficients = (ctypes.c_float * 3)(*dga.QUINTIC)
    call = dga.lib().dga_orthogonalize

    def work(G, out, workspace, stream):
        *batch, rows, cols = G.shape
        args = (dga.F32, dga.F32, batch[0] if batch else 1, rows, cols, G.data_ptr(), cols, rows * cols, out.data_ptr(), cols, rows * cols,
                1, coefficients, 1e-7, workspace.data_ptr(), workspace.numel(), stream.cuda_stream)
        torch.cuda.set_device(G.device)
        start.wait()
        seen = {call(*args) for _ in range(4000)}
        codes.append((seen, dga.dga_last_cuda_error()))

    threads, kept = [], []
    for i in (0, 1, 0, 1):
        G, out = inputs[i], torch.empty_like(inputs[i])
        size = dga.dga_orthogonalize_workspace_size(dga.F32, G.numel() // (G.shape[-1] * G.shape[-2]), *G.shape[-2:])
        kept.append((G, out, torch.empty(size, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
        threads.append(threading.Thread(target=work, args=kept[-1]))
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert [seen for seen, _ in codes] == [{dga.OK}] * 4, codes
    for (G, out, _, _), w in zip(kept, [dga.orthogonalize(inputs[i], steps=1) for i in (0, 1, 0, 1)]):
        assert torch.equal(out, w)


def test_host_threads_with_few_row_products_of_other_widths():
    """The same of the few-row products, whose shared memory goes by the width."""
    widths, K = (2432, 4864, 304, 9000), 256
    g = torch.Generator().manual_seed(6)
    x = torch.randn(4, K, generator=g).bfloat16().cuda()
    weights = [torch.randn(n, K, generator=g).bfloat16().cuda() for n in widths]
    want = [dga.gemm(x, w.t(), path=dga.PATH_SKINNY) for w in weights]
    codes, start = [], threading.Barrier(len(widths))
    one, zero = ctypes.c_float(1.0), ctypes.c_float(0.0)
    call = dga.lib().dga_gemm_general

    def work(w, out, stream):
        args = (dga.BF16, dga.BF16, dga.ROW_MAJOR, dga.COL_MAJOR, 4, w.shape[0], K, ctypes.byref(one), x.data_ptr(), K, w.data_ptr(), K,
                ctypes.byref(zero), out.data_ptr(), w.shape[0], None, None, 0, dga.PATH_SKINNY, stream.cuda_stream)
        torch.cuda.set_device(w.device)
        start.wait()
        codes.append({call(*args) for _ in range(6000)})

    kept = [(w, torch.empty_like(y), torch.cuda.Stream()) for w, y in zip(weights, want)]
    threads = [threading.Thread(target=work, args=k) for k in kept]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{dga.OK}] * len(widths)
    assert all(torch.equal(out, w) for (_, out, _), w in zip(kept, want))


def test_calls_run_on_their_tensors_device(monkeypatch):
    """With another device current, a call switches to its tensors' for its own
    duration (the other device is made up: its number is what the library's
    callers see as the current one)."""
    x = torch.randn(20, 64, generator=torch.Generator().manual_seed(3)).cuda()
    W = dga.mx_quantize(x)
    rows = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    cols, vals, v = torch.tensor([1, 0], dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda"), torch.ones(2, device="cuda")
    calls = [lambda: dga.mx_quantize(x).codes, lambda: dga.mx_dequantize(W), lambda: dga.mx_gemm(W, W), lambda: dga.mx_linear_forward(x, W),
             lambda: dga.mx_linear_backward(x, x, x @ x.t())[0], lambda: dga.orthogonalize(x), lambda: dga.gemm(x, x.t()),
             lambda: dga.sum_rows(x), lambda: dga.spmv_csr(rows, cols, vals, v)]
    want = [call() for call in calls]
    here, entered = x.device.index, []
    state = {"device": here + 1}

    class Device:
        def __init__(self, device):
            self.index = torch.device(device).index

        def __enter__(self):
            self.before, state["device"] = state["device"], self.index
            entered.append(self.index)

        def __exit__(self, *_):
            state["device"] = self.before

    monkeypatch.setattr(dga, "_current_device", lambda: state["device"], raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    for call, w in zip(calls, want):
        del entered[:]
        got = call()
        assert entered and set(entered) == {here}
        assert torch.equal(got, w)
    state["device"] = here
    for call in calls:
        del entered[:]
        call()
        assert not entered


@pytest.mark.parametrize("shape", [(3, 60, 70), (3, 100, 500), (3, 70, 2000), (3, 300, 140), (40, 300, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-40])
def test_a_zero_update_gives_zero_whatever_eps(dtype, shape, eps):
    G = torch.randn(*shape, generator=torch.Generator().manual_seed(5)).to(dtype)
    G[1] = 0.0
    got = dga.orthogonalize(G.cuda(), eps=eps)
    _sync_ok()
    assert not got[1].any()
    assert torch.equal(got[0], dga.orthogonalize(G[:1].expand(shape[0], *shape[1:]).contiguous().cuda(), eps=eps)[0])
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("fmt", FMT)
def test_gradients_of_a_column_major_output_gradient(fmt):
    x, w = (torch.randn(r, 70, generator=torch.Generator().manual_seed(r)).cuda() for r in (50, 90))
    g = torch.randn(50, 90, generator=torch.Generator().manual_seed(7)).cuda()
    want = dga.mx_linear_backward(x, w, g, fmt)
    got = dga.mx_linear_backward(x, w, g.t().contiguous().t(), fmt)
    _sync_ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("T", [7, 40, 300])
def test_chains_in_a_graph(fmt, T):
    """Quantisation and back, the layer and both its gradients, captured and
    replayed on new inputs."""
    def values(seed, rows, cols):
        return torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed)).cuda()
    x, w, g = values(1, T, 200), values(2, 150, 200), values(3, T, 150)

    def chain():
        W = dga.mx_quantize(w, fmt)
        back = dga.mx_dequantize(dga.mx_quantize(x, fmt, transpose=True))
        return (back, dga.mx_linear_forward(x, W), *dga.mx_linear_backward(x, w, g, fmt))

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for t, seed in ((x, 11), (w, 12), (g, 13)):
        t.copy_(values(seed, *t.shape))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    _sync_ok()
    for got, want in zip(out, chain()):
        assert torch.equal(got, want)


@pytest.mark.parametrize("T,N,K", [(5, 130, 300), (16, 300, 1000), (17, 300, 257), (200, 140, 520), (300, 260, 800)])
def test_products_with_factors_that_are_no_powers_of_two(T, N, K):
    """The product and the layer against fp64 products of the values their codes
    stand for.  Beside the sums' bound: alpha times both factors, and each
    operand's scale times factor and that times code, are rounded to fp32: six
    roundings of 2^-24, doubled."""
    g = torch.Generator().manual_seed(T)
    x, w = torch.randn(T, K, generator=g), torch.randn(N, K, generator=g) / K ** 0.5
    fx, fw = (torch.tensor([float(t.abs().max()) / 2688.0], device="cuda") for t in (x, w))
    X, W = dga.mx_quantize(x.cuda(), dga.NVFP4, tensor_scale=fx), dga.mx_quantize(w.cuda(), dga.NVFP4, tensor_scale=fw)
    A, B = dga.mx_dequantize(X).cpu().double().numpy(), dga.mx_dequantize(W).cpu().double().numpy()
    want = A @ B.T
    tol = ref.product_bound(A, B, K) + 12 * 2.0 ** -24 * (np.abs(A) @ np.abs(B).T) + np.abs(want) * 2.0 ** -23
    y = dga.mx_linear_forward(x.cuda(), W, tensor_scale=fx)
    p = dga.mx_gemm(X, W, out_dtype=dga.F32)
    _sync_ok()
    assert torch.equal(y, p)
    assert (np.abs(p.cpu().double().numpy() - want) <= tol).all()


def _inside(rows, cols, dtype, left):
    """(memory, its part rows x cols) with 24 columns or more on the right, rows
    above and below, and rows that start on 16 bytes (for left = 0 or 8)."""
    memory = torch.full((rows + 8, cols + -cols % 8 + 32), 7.0, dtype=dtype, device="cuda")
    return memory, memory[4:4 + rows, left:left + cols]


@pytest.mark.parametrize("left", [0, 3, 8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(3, 77), (100, 505), (300, 505), (700, 131), (600, 1021), (600, 1028)])
def test_products_leave_what_is_beside_c(M, N, dtype, left):
    """Results whose rows start on 16 bytes and end anywhere."""
    g = torch.Generator().manual_seed(N)
    a, b = torch.randn(M, 200, generator=g).cuda(), torch.randn(N, 200, generator=g).cuda()
    A, B = dga.mx_quantize(a), dga.mx_quantize(b)
    memory, C = _inside(M, N, dtype, left)
    dga.mx_gemm(A, B, C)
    _sync_ok()
    assert torch.equal(C, dga.mx_gemm(A, B, out_dtype=OUT[dtype]))
    C.fill_(7.0)
    assert bool((memory == 7.0).all())
    memory, Y = _inside(M, N, dtype, left)
    dga.mx_linear_forward(a, B, Y=Y)
    _sync_ok()
    Y.fill_(7.0)
    assert bool((memory == 7.0).all())


@pytest.mark.parametrize("left", [0, 3, 8])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch,m,n", [(2, 60, 77), (1, 140, 333), (1, 333, 140), (1, 200, 1003), (3, 300, 333), (3, 333, 301), (10, 630, 1482),
                                       (10, 1482, 630), (2, 1100, 1100)])
def test_updates_leave_what_is_beside_the_result(batch, m, n, dtype, left):
    G = torch.randn(batch, m, n, generator=torch.Generator().manual_seed(m)).to(dtype).cuda()
    memory, O = _inside(batch * m, n, dtype, left)
    O = O.unflatten(0, (batch, m))
    dga.orthogonalize(G, out=O)
    _sync_ok()
    assert torch.equal(O, dga.orthogonalize(G))
    O.fill_(7.0)
    assert bool((memory == 7.0).all())


def test_gradients_leave_what_is_beside_them():
    """The C call's own leading dimensions of both gradients."""
    T, N, K = 520, 300, 397
    g = torch.Generator().manual_seed(9)
    x, w, d = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((T, K), (N, K), (T, N)))
    want = dga.mx_linear_backward(x, w, d, dga.MXFP4)
    memory_x, dX = _inside(T, K, torch.bfloat16, 8)
    memory_w, dW = _inside(N, K, torch.bfloat16, 0)
    size = dga.dga_mx_linear_backward_workspace_size(dga.MXFP4, T, N, K)
    workspace = torch.empty(size, dtype=torch.uint8, device="cuda")
    st = dga.dga_mx_linear_backward(dga.MXFP4, dga.BF16, dga.BF16, dga.BF16, T, N, K, x.data_ptr(), K, None, w.data_ptr(), K, None,
                                    d.data_ptr(), N, None, dX.data_ptr(), dX.stride(0), dW.data_ptr(), dW.stride(0), None,
                                    workspace.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert st == dga.OK
    _sync_ok()
    assert torch.equal(dX, want[0]) and torch.equal(dW, want[1])
    for memory, part in ((memory_x, dX), (memory_w, dW)):
        part.fill_(7.0)
        assert bool((memory == 7.0).all())
