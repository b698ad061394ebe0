// mx_api.cu -- the C entry points of the 4-bit microscaled matrices: argument
// checks, then the launches of mx_quant.cu and mx_gemm.cu on the caller's
// stream.  Errors are reported as in api.cu: -(1-based position).
#include <cuda_runtime.h>

#include "dga_internal.h"
#include "mx_common.cuh"

using namespace dga;

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 30;  // the kernels count rows, bytes and scales in 31 bits

bool format_ok(int format) { return format == DGA_MXFP4 || format == DGA_NVFP4; }
bool float_type(int t) { return t == DGA_F32 || t == DGA_BF16 || t == DGA_F16; }
int64_t type_size(int t) { return t == DGA_F32 ? 4 : 2; }
int64_t at_least_one(int64_t x) { return x > 1 ? x : 1; }

struct Span {
    uintptr_t lo, hi;
};
Span span(const void* p, int64_t rows, int64_t stride_bytes, int64_t row_bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>((rows - 1) * stride_bytes + row_bytes)};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

int64_t scales_bytes(int format, int64_t rows, int64_t K) {
    return (rows + 127) / 128 * mx_tiles_k(format, K) * kMxTileBytes;
}
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// A 4-bit matrix's pointers: position of the first wrong argument (codes at
// `pos`, then ld, scales, factor), or 0.
int check_matrix(int format, int64_t K, const void* codes, int64_t ld, const void* scales, const float* factor,
                 int pos) {
    if (!codes || !aligned(codes, 16)) return pos;
    if (ld < mx_row_bytes(K) || ld % 16 != 0) return pos + 1;
    if (!scales || !aligned(scales, 16)) return pos + 2;
    if (factor && format == DGA_MXFP4) return pos + 3;
    return 0;
}

int device(DeviceInfo* dev) {
    cudaError_t e = current_device_info(dev);
    if (e != cudaSuccess) return note_cuda_error(e);
    return dev->major == 10 && dev->minor == 3 ? DGA_OK : DGA_ERR_DEVICE;
}

// rows x K in 4 bits inside a workspace: codes, then scales.
int64_t held_bytes(int format, int64_t rows, int64_t K) {
    return round_up(rows * mx_row_bytes(K), 256) + scales_bytes(format, rows, K);
}
MxMatrix held_at(uint8_t* ws, int64_t rows, int64_t K, const float* factor) {
    return {ws, mx_row_bytes(K), ws + round_up(rows * mx_row_bytes(K), 256), factor};
}

}  // namespace

extern "C" {

int64_t dga_mx_row_bytes(int64_t K) { return K > 0 ? mx_row_bytes(K) : 0; }

size_t dga_mx_scales_size(dga_mx_format format, int64_t rows, int64_t K) {
    if (!format_ok(format) || rows <= 0 || K <= 0) return 0;
    return static_cast<size_t>(scales_bytes(format, rows, K));
}

int dga_mx_quantize(dga_mx_format format, dga_dtype in_dtype, int transpose, int64_t rows, int64_t cols,
                    const void* X, int64_t ldx, const float* tensor_scale, void* codes, int64_t ld_codes,
                    void* scales, dga_stream_t stream) {
    if (!format_ok(format) || !float_type(in_dtype)) return DGA_ERR_UNSUPPORTED;
    if (transpose != 0 && transpose != 1) return -3;
    if (rows < 0 || rows >= kMaxDim) return -4;
    if (cols < 0 || cols >= kMaxDim) return -5;
    if (tensor_scale && format == DGA_MXFP4) return -8;
    set_last_launches(0);
    if (rows == 0 || cols == 0) return DGA_OK;
    if (!X) return -6;
    if (ldx < at_least_one(cols)) return -7;
    const int64_t R = transpose ? cols : rows, K = transpose ? rows : cols;
    const int bad = check_matrix(format, K, codes, ld_codes, scales, nullptr, 9);
    if (bad) return -bad;
    const Span x = span(X, rows, ldx * type_size(in_dtype), cols * type_size(in_dtype));
    const Span c = span(codes, R, ld_codes, mx_row_bytes(K));
    const Span s = span(scales, 1, 0, scales_bytes(format, R, K));
    if (meet(x, c) || meet(x, s) || meet(c, s)) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    MxQuantArgs a{format, in_dtype, transpose != 0, rows, cols, X, ldx, tensor_scale, static_cast<uint8_t*>(codes),
                  ld_codes, static_cast<uint8_t*>(scales), reinterpret_cast<cudaStream_t>(stream)};
    const cudaError_t e = mx_quantize_launch(a, dev);
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(1);
    return DGA_OK;
}

int dga_mx_dequantize(dga_mx_format format, dga_dtype out_dtype, int64_t rows, int64_t cols, const void* codes,
                      int64_t ld_codes, const void* scales, const float* tensor_scale, void* Y, int64_t ldy,
                      dga_stream_t stream) {
    if (!format_ok(format) || !float_type(out_dtype)) return DGA_ERR_UNSUPPORTED;
    if (rows < 0 || rows >= kMaxDim) return -3;
    if (cols < 0 || cols >= kMaxDim) return -4;
    set_last_launches(0);
    if (rows == 0 || cols == 0) return DGA_OK;
    const int bad = check_matrix(format, cols, codes, ld_codes, scales, tensor_scale, 5);
    if (bad) return -bad;
    if (!Y) return -9;
    if (ldy < at_least_one(cols)) return -10;
    const Span y = span(Y, rows, ldy * type_size(out_dtype), cols * type_size(out_dtype));
    if (meet(y, span(codes, rows, ld_codes, mx_row_bytes(cols))) ||
        meet(y, span(scales, 1, 0, scales_bytes(format, rows, cols))))
        return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    const MxMatrix q{codes, ld_codes, scales, tensor_scale};
    const cudaError_t e = mx_dequantize_launch(format, out_dtype, q, rows, cols, Y, ldy, dev,
                                               reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(1);
    return DGA_OK;
}

int dga_mx_gemm(dga_mx_format format, dga_dtype out_dtype, int64_t M, int64_t N, int64_t K, const float* alpha,
                const void* A_codes, int64_t lda, const void* A_scales, const float* A_tensor_scale,
                const void* B_codes, int64_t ldb, const void* B_scales, const float* B_tensor_scale,
                const float* beta, void* C, int64_t ldc, const void* bias, dga_stream_t stream) {
    if (!format_ok(format) || !float_type(out_dtype)) return DGA_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim) return -3;
    if (N < 0 || N >= kMaxDim) return -4;
    if (K < 0 || K >= kMaxDim) return -5;
    if (!alpha) return -6;
    if (!beta) return -15;
    set_last_launches(0);
    if (M == 0 || N == 0) return DGA_OK;
    const bool reads = K > 0 && *alpha != 0.0f;
    if (reads) {
        int bad = check_matrix(format, K, A_codes, lda, A_scales, A_tensor_scale, 7);
        if (!bad) bad = check_matrix(format, K, B_codes, ldb, B_scales, B_tensor_scale, 11);
        if (bad) return -bad;
    }
    if (!C) return -16;
    if (ldc < at_least_one(N)) return -17;
    const int64_t es = type_size(out_dtype);
    const Span c = span(C, M, ldc * es, N * es);
    if (bias && meet(c, span(bias, 1, 0, N * es))) return DGA_ERR_OVERLAP;
    if (reads && (meet(c, span(A_codes, M, lda, mx_row_bytes(K))) || meet(c, span(B_codes, N, ldb, mx_row_bytes(K))) ||
                  meet(c, span(A_scales, 1, 0, scales_bytes(format, M, K))) ||
                  meet(c, span(B_scales, 1, 0, scales_bytes(format, N, K)))))
        return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    MxGemmArgs a{format, out_dtype, M, N, K, *alpha, *beta, {A_codes, lda, A_scales, A_tensor_scale},
                 {B_codes, ldb, B_scales, B_tensor_scale}, C, ldc, bias, false,
                 reinterpret_cast<cudaStream_t>(stream), nullptr, 0, 0};
    int launches = 0;
    const cudaError_t e = mx_gemm_launch(a, dev, &launches);
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

size_t dga_mx_linear_workspace_size(dga_mx_format format, int64_t M, int64_t K) {
    if (!format_ok(format) || M <= kMxFusedRows || K <= 0) return 0;
    return static_cast<size_t>(round_up(M * mx_row_bytes(K), 256) + scales_bytes(format, M, K));
}

int dga_mx_linear(dga_mx_format format, dga_dtype x_dtype, dga_dtype out_dtype, int64_t M, int64_t N, int64_t K,
                  const void* X, int64_t ldx, const float* x_tensor_scale, const void* W_codes, int64_t ldw,
                  const void* W_scales, const float* W_tensor_scale, const void* bias, void* Y, int64_t ldy,
                  void* workspace, size_t workspace_bytes, dga_stream_t stream) {
    if (!format_ok(format) || !float_type(x_dtype) || !float_type(out_dtype)) return DGA_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim) return -4;
    if (N < 0 || N >= kMaxDim) return -5;
    if (K < 0 || K >= kMaxDim) return -6;
    set_last_launches(0);
    if (M == 0 || N == 0) return DGA_OK;
    const size_t need = dga_mx_linear_workspace_size(format, M, K);
    if (K > 0) {
        if (!X) return -7;
        if (ldx < at_least_one(K)) return -8;
        if (x_tensor_scale && format == DGA_MXFP4) return -9;
        const int bad = check_matrix(format, K, W_codes, ldw, W_scales, W_tensor_scale, 10);
        if (bad) return -bad;
        if (need > 0 && workspace && !aligned(workspace, 16)) return -17;
        if (workspace_bytes > 0 && !workspace) return -17;
        if (workspace_bytes < need) return DGA_ERR_WORKSPACE;
    }
    if (!Y) return -15;
    if (ldy < at_least_one(N)) return -16;
    const int64_t es = type_size(out_dtype);
    const Span y = span(Y, M, ldy * es, N * es);
    if (bias && meet(y, span(bias, 1, 0, N * es))) return DGA_ERR_OVERLAP;
    const float one = 1.0f, zero = 0.0f;
    if (K == 0)
        return dga_mx_gemm(format, out_dtype, M, N, 0, &one, nullptr, 0, nullptr, nullptr, nullptr, 0, nullptr, nullptr,
                           &zero, Y, ldy, bias, stream);
    const Span w = span(workspace, 1, 0, static_cast<int64_t>(need));
    const Span wc = span(W_codes, N, ldw, mx_row_bytes(K)), wsc = span(W_scales, 1, 0, scales_bytes(format, N, K));
    const Span x = span(X, M, ldx * type_size(x_dtype), K * type_size(x_dtype));
    if (meet(y, x) || meet(y, wc) || meet(y, wsc) ||
        (need > 0 && (meet(y, w) || meet(w, x) || meet(w, wc) || meet(w, wsc) || (bias && meet(w, span(bias, 1, 0, N * es))))))
        return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    MxGemmArgs a{format, out_dtype, M, N, K, 1.0f, 0.0f, {nullptr, 0, nullptr, x_tensor_scale},
                 {W_codes, ldw, W_scales, W_tensor_scale}, Y, ldy, bias, false, s, X, ldx, x_dtype};
    cudaError_t e;
    int launches = 0;
    if (M > kMxFusedRows) {
        uint8_t* codes = static_cast<uint8_t*>(workspace);
        uint8_t* scales = codes + round_up(M * mx_row_bytes(K), 256);
        MxQuantArgs q{format, x_dtype, false, M, K, X, ldx, x_tensor_scale, codes, mx_row_bytes(K), scales, s};
        e = mx_quantize_launch(q, dev);
        if (e != cudaSuccess) return note_cuda_error(e);
        launches = 1;
        a.A = {codes, mx_row_bytes(K), scales, x_tensor_scale};
        a.after_quantize = true;
        a.X = nullptr;
    }
    e = mx_gemm_launch(a, dev, &launches);
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

size_t dga_mx_linear_backward_workspace_size(dga_mx_format format, int64_t M, int64_t N, int64_t K) {
    if (!format_ok(format) || M <= 0 || N <= 0 || K <= 0) return 0;
    return static_cast<size_t>(held_bytes(format, M, N) + held_bytes(format, K, N) + held_bytes(format, N, M) +
                               held_bytes(format, K, M));
}

int dga_mx_linear_backward(dga_mx_format format, dga_dtype x_dtype, dga_dtype w_dtype, dga_dtype g_dtype, int64_t M,
                           int64_t N, int64_t K, const void* X, int64_t ldx, const float* x_tensor_scale, const void* W,
                           int64_t ldw, const float* w_tensor_scale, const void* G, int64_t ldg,
                           const float* g_tensor_scale, void* dX, int64_t lddx, void* dW, int64_t lddw, float* db,
                           void* workspace, size_t workspace_bytes, dga_stream_t stream) {
    if (!format_ok(format) || !float_type(x_dtype) || !float_type(w_dtype) || !float_type(g_dtype)) return DGA_ERR_UNSUPPORTED;
    if (M < 0 || M >= kMaxDim) return -5;
    if (N < 0 || N >= kMaxDim) return -6;
    if (K < 0 || K >= kMaxDim) return -7;
    if (x_tensor_scale && format == DGA_MXFP4) return -10;
    if (w_tensor_scale && format == DGA_MXFP4) return -13;
    if (g_tensor_scale && format == DGA_MXFP4) return -16;
    set_last_launches(0);
    const bool has_x = M > 0 && K > 0, has_w = N > 0 && K > 0, has_g = M > 0 && N > 0;
    if (has_x && (!X || ldx < K)) return !X ? -8 : -9;
    if (has_w && (!W || ldw < K)) return !W ? -11 : -12;
    if (has_g && (!G || ldg < N)) return !G ? -14 : -15;
    if (has_x && (!dX || lddx < K)) return !dX ? -17 : -18;
    if (has_w && (!dW || lddw < K)) return !dW ? -19 : -20;
    const size_t need = dga_mx_linear_backward_workspace_size(format, M, N, K);
    if (workspace && !aligned(workspace, 256)) return -22;
    if (workspace_bytes > 0 && !workspace) return -22;
    if (workspace_bytes < need) return DGA_ERR_WORKSPACE;
    const int64_t gs = type_size(g_dtype);
    // what is read, then what is written
    Span spans[7];
    int n = 0;
    auto matrix = [&](bool there, const void* p, int64_t rows, int64_t ld, int64_t cols, int64_t es) {
        if (there) spans[n++] = span(p, rows, ld * es, cols * es);
    };
    matrix(has_x, X, M, ldx, K, type_size(x_dtype));
    matrix(has_w, W, N, ldw, K, type_size(w_dtype));
    matrix(has_g, G, M, ldg, N, gs);
    const int inputs = n;
    matrix(has_x, dX, M, lddx, K, gs);
    matrix(has_w, dW, N, lddw, K, gs);
    matrix(db != nullptr && N > 0, db, 1, N, N, 4);
    matrix(need > 0, workspace, 1, static_cast<int64_t>(need), static_cast<int64_t>(need), 1);
    for (int i = inputs; i < n; ++i)
        for (int j = 0; j < i; ++j)
            if (meet(spans[i], spans[j])) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int launches = 0;
    cudaError_t e = cudaSuccess;
    // rows x K in 4 bits, of T's rows or (transposed) its columns
    auto quantise = [&](int dtype, bool transpose, const void* T, int64_t ld, int64_t rows, int64_t k, const float* factor) {
        const MxMatrix q = held_at(ws, rows, k, factor);
        ws += held_bytes(format, rows, k);
        if (e != cudaSuccess) return q;
        MxQuantArgs a{format, dtype, transpose, transpose ? k : rows, transpose ? rows : k, T, ld, factor,
                      static_cast<uint8_t*>(const_cast<void*>(q.codes)), q.ld, static_cast<uint8_t*>(const_cast<void*>(q.scales)), s};
        e = mx_quantize_launch(a, dev);
        if (e == cudaSuccess) ++launches;
        return q;
    };
    // C (rows x cols) <- P Q^T, zero for k == 0
    auto product = [&](const MxMatrix& P, const MxMatrix& Q, int64_t rows, int64_t cols, int64_t k, void* C, int64_t ldc) {
        if (e != cudaSuccess || rows == 0 || cols == 0) return;
        MxGemmArgs a{format, g_dtype, rows, cols, k, 1.0f, 0.0f, P, Q, C, ldc, nullptr, false, s, nullptr, 0, 0};
        int l = 0;
        e = mx_gemm_launch(a, dev, &l);
        launches += l;
    };
    MxMatrix g{}, w{}, gt{}, xt{};
    if (need > 0) {
        g = quantise(g_dtype, false, G, ldg, M, N, g_tensor_scale);
        w = quantise(w_dtype, true, W, ldw, K, N, w_tensor_scale);
        gt = quantise(g_dtype, true, G, ldg, N, M, g_tensor_scale);
        xt = quantise(x_dtype, true, X, ldx, K, M, x_tensor_scale);
    }
    product(g, w, M, K, N, dX, lddx);
    product(gt, xt, N, K, M, dW, lddw);
    if (e == cudaSuccess && db && N > 0) {
        e = sum_rows_launch(g_dtype, M, N, G, ldg, db, s);
        if (e == cudaSuccess) ++launches;
    }
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

}  // extern "C"
