// gated_api.cu -- the C entry points of the gated feed-forward layer and of
// 4-bit weights with group scales: argument checks, then the launches on the
// caller's stream.  Errors are reported as in api.cu: -(1-based position).
#include <cuda_runtime.h>

#include <algorithm>

#include "dga_internal.h"
#include "mx_common.cuh"

using namespace dga;

namespace {

constexpr int64_t kMaxDim = int64_t{1} << 30;

bool float_type(int t) { return t == DGA_F32 || t == DGA_BF16 || t == DGA_F16; }
bool half_type(int t) { return t == DGA_BF16 || t == DGA_F16; }
bool act_ok(int a) { return a >= DGA_SILU && a <= DGA_SIGMOID; }
bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }
int64_t type_size(int t) { return t == DGA_F32 ? 4 : 2; }
int64_t at_least_one(int64_t x) { return x > 1 ? x : 1; }
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
bool dim_ok(int64_t x) { return x >= 0 && x < kMaxDim; }

// Arrays that a call reads and writes, to find those that meet.
struct Arrays {
    struct Span {
        uintptr_t lo, hi;
    };
    Span read[8], written[6];
    int reads = 0, writes = 0;

    static Span of(const void* p, int64_t rows, int64_t stride_bytes, int64_t row_bytes) {
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        return {lo, lo + static_cast<uintptr_t>((rows - 1) * stride_bytes + row_bytes)};
    }
    void in(const void* p, int64_t rows, int64_t stride_bytes, int64_t row_bytes) {
        if (p && rows > 0 && row_bytes > 0) read[reads++] = of(p, rows, stride_bytes, row_bytes);
    }
    void out(const void* p, int64_t rows, int64_t stride_bytes, int64_t row_bytes) {
        if (p && rows > 0 && row_bytes > 0) written[writes++] = of(p, rows, stride_bytes, row_bytes);
    }
    bool meet() const {
        auto both = [](const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; };
        for (int i = 0; i < writes; ++i) {
            for (int j = 0; j < reads; ++j)
                if (both(written[i], read[j])) return true;
            for (int j = 0; j < i; ++j)
                if (both(written[i], written[j])) return true;
        }
        return false;
    }
};

int device(DeviceInfo* dev) {
    cudaError_t e = current_device_info(dev);
    if (e != cudaSuccess) return note_cuda_error(e);
    return dev->major == 10 && dev->minor == 3 ? DGA_OK : DGA_ERR_DEVICE;
}

const char aligned_probe[16] __attribute__((aligned(16))) = {};

// C (M x N, out type) = op(A) op(B) + bias, as gemm_run takes it; with no
// pointers given, for its workspace's size.
GemmArgs product(int in, int out, int layout_a, int layout_b, int64_t M, int64_t N, int64_t K, const void* A, int64_t lda,
                 const void* B, int64_t ldb, void* C, int64_t ldc, const void* bias, cudaStream_t s) {
    GemmArgs g{};
    g.in_dtype = in;
    g.out_dtype = out;
    g.layout_a = layout_a;
    g.layout_b = layout_b;
    g.M = M, g.N = N, g.K = K;
    g.alpha_f = 1.0f;
    g.A = A ? A : aligned_probe;
    g.lda = at_least_one(lda);
    g.B = B ? B : aligned_probe;
    g.ldb = at_least_one(ldb);
    g.C = C;
    g.ldc = ldc;
    g.bias = bias;
    g.stream = s;
    g.deep = 1;
    return g;
}

// P as fp32, rows of whole 16 bytes, inside a workspace.
int64_t held_ld(int64_t F) { return round_up(2 * F, 4); }
int64_t held_bytes(int64_t M, int64_t F) { return round_up(M * held_ld(F) * 4, 256); }

// Scratch of dga_gated.  16-bit types: X and W in rows that start on 16 bytes,
// where they have none.  fp32, and K = 0: P where the caller keeps none in fp32,
// the product's own.
struct ForwardPlan {
    bool fused;
    int64_t x, w, held, gemm;
    int64_t total() const { return x + w + held + gemm; }
};
ForwardPlan forward_plan(int dtype, int64_t M, int64_t F, int64_t K, int64_t ldx, int64_t ldw, bool save, const void* X,
                         const void* W) {
    ForwardPlan pl{};
    pl.fused = dtype != DGA_F32 && K > 0;
    if (pl.fused) {
        const int64_t row = round_up(K, 8) * 2;
        if (ldx % 8 != 0 || (X && !aligned(X, 16))) pl.x = round_up(M * row, 256);
        if (ldw % 8 != 0 || (W && !aligned(W, 16))) pl.w = round_up(2 * F * row, 256);
        return pl;
    }
    const bool direct = dtype == DGA_F32 && save;
    pl.held = direct ? 0 : held_bytes(M, F);
    pl.gemm = static_cast<int64_t>(gemm_wanted(product(dtype, DGA_F32, DGA_ROW_MAJOR, DGA_COL_MAJOR, M, 2 * F, K, X, ldx, W,
                                                       ldw, nullptr, 2 * F, nullptr, nullptr)));
    return pl;
}

// Scratch of dga_gated_backward: dP, the column sums' slices, the products' own.
struct BackwardPlan {
    int64_t ldd, dp, sums, gemm;
    int64_t total() const { return dp + sums + gemm; }
};
BackwardPlan backward_plan(int dtype, int64_t M, int64_t F, int64_t K, int64_t ldx, int64_t ldw, const void* X, const void* W) {
    BackwardPlan pl{};
    pl.ldd = round_up(2 * F, 16 / type_size(dtype));
    pl.dp = round_up(M * pl.ldd * type_size(dtype), 256);
    pl.sums = round_up(static_cast<int64_t>(gated_grad_partials(M, F)) * 4, 256);
    const size_t a = gemm_wanted(product(dtype, dtype, DGA_ROW_MAJOR, DGA_ROW_MAJOR, M, K, 2 * F, nullptr, pl.ldd, W, ldw, nullptr, K, nullptr, nullptr));
    const size_t b = gemm_wanted(product(dtype, dtype, DGA_COL_MAJOR, DGA_ROW_MAJOR, 2 * F, K, M, nullptr, pl.ldd, X, ldx, nullptr, K, nullptr, nullptr));
    pl.gemm = static_cast<int64_t>(std::max(a, b));
    return pl;
}

// A 4-bit weight's arguments: the position of the first wrong one (codes at
// `pos`, then ld, scales, ld, zeros, ld), or 0.
int check_q4(const Q4Matrix& q, int64_t K, int pos) {
    if (!q.codes || !aligned(q.codes, 16)) return pos;
    if (q.ld < mx_row_bytes(K) || q.ld % 16 != 0) return pos + 1;
    if (!q.scales || !aligned(q.scales, 2)) return pos + 2;
    const int64_t groups = (K + q.group - 1) / q.group;
    if (q.ld_scales < groups) return pos + 3;
    if (q.zeros && q.ld_zeros < groups) return pos + 5;
    return 0;
}
void q4_arrays(Arrays& a, const Q4Matrix& q, int64_t N, int64_t K, bool written) {
    const int64_t groups = (K + q.group - 1) / q.group;
    auto add = [&](const void* p, int64_t stride, int64_t row) { written ? a.out(p, N, stride, row) : a.in(p, N, stride, row); };
    add(q.codes, q.ld, mx_row_bytes(K));
    add(q.scales, q.ld_scales * 2, groups * 2);
    add(q.zeros, q.ld_zeros, groups);
}

// How a product on a 4-bit weight goes, and its scratch: X in rows that start on 16
// bytes, where a kernel needs them and it has none; the weight's values; a gated
// one's P (K = 0); the library's product's own.
//
//   rows    q4_rows, on the codes as they are: few rows.  8192 x 8192 in groups of 128,
//           32 rows: 24.5 us, q4_tc 22.4; 4096 x 4096: 8.7 and 10.0.  48 rows, 8192 x
//           8192: 45 and 23; 4096 x 4096: 12.7 and 10.4; 2048 x 2048: 5.4 and 7.2.
//   tensor  q4_tc, which makes the values as it goes, once for each 256 (gated: 128)
//           rows of X.  1024 rows of 8192 x 8192: 112 us, through the values 137;
//           2048: 223 and 201.  A gated one's values go to the fused layer:
//           8192 gate and up rows, K = 4096, 512 rows: 46 us on the codes, 63 through
//           the values; 1024: 90 and 65.
//   else the values are written out first.
struct Q4Plan {
    bool rows, tensor;
    int64_t ldv, x, values, held, gemm;
    int64_t total() const { return x + values + held + gemm; }
};
Q4Plan q4_plan(int dtype, int64_t M, int64_t N, int64_t K, int64_t ldx, bool gated, const void* X) {
    Q4Plan pl{};
    pl.ldv = round_up(K, 8);
    pl.rows = K > 0 && (M <= 32 || (M <= 64 && N * K <= (int64_t{1} << 22)));
    pl.tensor = K > 0 && !pl.rows && M <= (gated ? kQ4GatedTensorRows : kQ4TensorRows);
    if (pl.rows || pl.tensor || (gated && K > 0)) {
        if (ldx % 8 != 0 || (X && !aligned(X, 16))) pl.x = round_up(M * pl.ldv * 2, 256);
        if (!pl.rows && !pl.tensor) pl.values = round_up(N * pl.ldv * 2, 256);
        return pl;
    }
    pl.values = round_up(N * pl.ldv * 2, 256);
    pl.held = gated ? held_bytes(M, N / 2) : 0;
    pl.gemm = static_cast<int64_t>(gemm_wanted(product(dtype, gated ? DGA_F32 : dtype, DGA_ROW_MAJOR, DGA_COL_MAJOR, M, N, K, X,
                                                       ldx, nullptr, pl.ldv, nullptr, N, nullptr, nullptr)));
    return pl;
}

// Y, or (gated, N its outputs) the gated layer's result, by q4_rows, q4_tc or the gated
// layer's kernel on the values.
cudaError_t q4_by_kernel(const Q4Plan& pl, int dtype, int act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                         const Q4Matrix& q, const void* bias, void* Y, int64_t ldy, bool gated, uint8_t* ws, const DeviceInfo& dev,
                         cudaStream_t s, int* launches) {
    cudaError_t e = cudaSuccess;
    if (pl.x) {
        e = copy_rows_launch({M, K, X, ldx, ws, pl.ldv}, nullptr, s);
        if (e != cudaSuccess) return e;
        ++*launches;
        X = ws;
        ldx = pl.ldv;
    }
    if (pl.rows) {
        e = q4_rows_launch(dtype, act, M, N, K, X, ldx, q, bias, Y, ldy, gated, dev, s);
    } else if (pl.tensor) {
        e = q4_tc_launch(dtype, act, M, N, K, X, ldx, q, bias, Y, ldy, gated, dev, s);
    } else {
        e = q4_dequantize_launch(dtype, dtype, 2 * N, K, q, ws + pl.x, pl.ldv, s);
        if (e != cudaSuccess) return e;
        ++*launches;
        const GatedArgs g{dtype, act, M, N, K, X, ldx, ws + pl.x, pl.ldv, bias, Y, ldy, nullptr, 0, s};
        e = gated_tc_supports(g) ? gated_tc_launch(g, dev) : cudaErrorNotSupported;
    }
    if (e == cudaSuccess) ++*launches;
    return e;
}

// [X W^T + bias] of a 4-bit W through its values: into Y, or (gated) into P's place in the workspace.
cudaError_t q4_by_values(const Q4Plan& pl, int dtype, int out, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx,
                         const Q4Matrix& q, const void* bias, void* Y, int64_t ldy, uint8_t* ws, const DeviceInfo& dev,
                         cudaStream_t s, int* launches) {
    cudaError_t e = cudaSuccess;
    if (K > 0) {
        e = q4_dequantize_launch(dtype, dtype, N, K, q, ws, pl.ldv, s);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    GemmArgs g = product(dtype, out, DGA_ROW_MAJOR, DGA_COL_MAJOR, M, N, K, X, ldx, ws, pl.ldv, Y, ldy, bias, s);
    g.ws = ws + pl.values + pl.held;
    g.ws_bytes = static_cast<size_t>(pl.gemm);
    return gemm_run(g, dev, launches);
}

}  // namespace

extern "C" {

size_t dga_gated_workspace_size(dga_dtype dtype, int64_t M, int64_t F, int64_t K, int64_t ldx, int64_t ldw, int save) {
    if (!float_type(dtype) || M <= 0 || F <= 0 || K < 0 || !dim_ok(M) || !dim_ok(F) || !dim_ok(K)) return 0;
    const ForwardPlan pl = forward_plan(dtype, M, F, K, ldx, ldw, save != 0, nullptr, nullptr);
    return static_cast<size_t>(pl.total());
}

int dga_gated(dga_dtype dtype, dga_activation act, int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx, const void* W,
              int64_t ldw, const void* bias, void* H, int64_t ldh, void* P, int64_t ldp, void* workspace,
              size_t workspace_bytes, dga_stream_t stream) {
    if (!float_type(dtype) || !act_ok(act)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(M)) return -3;
    if (!dim_ok(F)) return -4;
    if (!dim_ok(K)) return -5;
    set_last_launches(0);
    if (M == 0 || F == 0) return DGA_OK;
    const int64_t es = type_size(dtype);
    if (K > 0 && (!X || !aligned(X, es))) return -6;
    if (ldx < at_least_one(K)) return -7;
    if (K > 0 && (!W || !aligned(W, es))) return -8;
    if (ldw < at_least_one(K)) return -9;
    if (bias && !aligned(bias, es)) return -10;
    if (!H || !aligned(H, es)) return -11;
    if (ldh < F) return -12;
    if (P && !aligned(P, es)) return -13;
    if (P && ldp < 2 * F) return -14;
    if ((workspace_bytes > 0 && !workspace) || (workspace && !aligned(workspace, 16))) return -15;
    const ForwardPlan pl = forward_plan(dtype, M, F, K, ldx, ldw, P != nullptr, X, W);
    const int64_t need = pl.total();
    if (workspace_bytes < static_cast<size_t>(need)) return DGA_ERR_WORKSPACE;
    Arrays a;
    if (K > 0) a.in(X, M, ldx * es, K * es), a.in(W, 2 * F, ldw * es, K * es);
    a.in(bias, 1, 0, 2 * F * es);
    a.out(H, M, ldh * es, F * es);
    a.out(P, M, ldp * es, 2 * F * es);
    a.out(workspace, 1, 0, need);
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (pl.fused) {
        GatedArgs g{dtype, act, M, F, K, X, ldx, W, ldw, bias, H, ldh, P, ldp, s};
        const int64_t ld = round_up(K, 8);
        if (pl.x || pl.w) {
            const CopyRows x{M, K, X, ldx, ws, ld}, w{2 * F, K, W, ldw, ws + pl.x, ld};
            e = pl.x ? copy_rows_launch(x, pl.w ? &w : nullptr, s) : copy_rows_launch(w, nullptr, s);
            if (pl.x) g.X = x.Y, g.ldx = ld;
            if (pl.w) g.W = w.Y, g.ldw = ld;
            ++launches;
        }
        if (e == cudaSuccess)
            e = gated_skinny_supports(g) ? gated_skinny_launch(g, dev) : gated_tc_supports(g) ? gated_tc_launch(g, dev) : cudaErrorNotSupported;
        if (e != cudaSuccess) return note_cuda_error(e);
        set_last_launches(launches + 1);
        return DGA_OK;
    }
    const bool direct = pl.held == 0;
    void* sums = direct ? P : ws;
    const int64_t lds = direct ? ldp : held_ld(F);
    // the bias is of the input type; a product with fp32 output of 16-bit
    // inputs takes an fp32 one, so it is added with the activation there
    GemmArgs g = product(dtype, DGA_F32, DGA_ROW_MAJOR, DGA_COL_MAJOR, M, 2 * F, K, X, ldx, W, ldw, sums, lds,
                         dtype == DGA_F32 ? bias : nullptr, s);
    g.ws = ws + pl.held;
    g.ws_bytes = static_cast<size_t>(pl.gemm);
    e = gemm_run(g, dev, &launches);
    if (e == cudaSuccess) {
        e = gated_act_launch(dtype, act, M, F, static_cast<const float*>(sums), lds, dtype == DGA_F32 ? nullptr : bias, H, ldh,
                             direct ? nullptr : P, ldp, s);
        if (e == cudaSuccess) ++launches;
    }
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

size_t dga_gated_backward_workspace_size(dga_dtype dtype, int64_t M, int64_t F, int64_t K, int64_t ldx, int64_t ldw) {
    if (!float_type(dtype) || F <= 0 || !dim_ok(M) || !dim_ok(F) || !dim_ok(K)) return 0;
    return static_cast<size_t>(backward_plan(dtype, M, F, K, ldx, ldw, nullptr, nullptr).total());
}

int dga_gated_backward(dga_dtype dtype, dga_activation act, int64_t M, int64_t F, int64_t K, const void* X, int64_t ldx,
                       const void* W, int64_t ldw, const void* P, int64_t ldp, const void* G, int64_t ldg, void* dX,
                       int64_t lddx, void* dW, int64_t lddw, float* db, void* workspace, size_t workspace_bytes,
                       dga_stream_t stream) {
    if (!float_type(dtype) || !act_ok(act)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(M)) return -3;
    if (!dim_ok(F)) return -4;
    if (!dim_ok(K)) return -5;
    set_last_launches(0);
    const int64_t es = type_size(dtype);
    const bool has_p = M > 0 && F > 0, has_x = M > 0 && K > 0, has_w = F > 0 && K > 0;
    auto bad = [&](const void* p) { return !p || !aligned(p, es); };
    if (has_x && dW && bad(X)) return -6;
    if (ldx < at_least_one(K)) return -7;
    if (has_w && dX && bad(W)) return -8;
    if (ldw < at_least_one(K)) return -9;
    if (has_p && bad(P)) return -10;
    if (ldp < at_least_one(2 * F)) return -11;
    if (has_p && bad(G)) return -12;
    if (ldg < at_least_one(F)) return -13;
    if (dX && !aligned(dX, es)) return -14;
    if (dX && lddx < at_least_one(K)) return -15;
    if (dW && !aligned(dW, es)) return -16;
    if (dW && lddw < at_least_one(K)) return -17;
    if (db && !aligned(db, 4)) return -18;
    if ((workspace_bytes > 0 && !workspace) || (workspace && !aligned(workspace, 256))) return -19;
    BackwardPlan pl{};
    if (F > 0) pl = backward_plan(dtype, M, F, K, ldx, ldw, X, W);
    if (workspace_bytes < static_cast<size_t>(pl.total())) return DGA_ERR_WORKSPACE;
    Arrays a;
    if (has_x) a.in(X, M, ldx * es, K * es), a.out(dX, M, lddx * es, K * es);
    if (has_w) a.in(W, 2 * F, ldw * es, K * es), a.out(dW, 2 * F, lddw * es, K * es);
    if (has_p) a.in(P, M, ldp * es, 2 * F * es), a.in(G, M, ldg * es, F * es);
    a.out(db, 1, 0, 2 * F * 4);
    a.out(workspace, 1, 0, pl.total());
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int launches = 0;
    cudaError_t e = cudaSuccess;
    if (F > 0 && (M > 0 || db))
        e = gated_grad_launch(dtype, act, M, F, P, ldp, G, ldg, ws, pl.ldd, db, reinterpret_cast<float*>(ws + pl.dp), s,
                              &launches);
    auto run = [&](int layout_a, int64_t rows, int64_t k, const void* B, int64_t ldb, void* C, int64_t ldc) {
        if (e != cudaSuccess || !C || rows == 0 || K == 0) return;
        GemmArgs g = product(dtype, dtype, layout_a, DGA_ROW_MAJOR, rows, K, k, ws, pl.ldd, B, ldb, C, ldc, nullptr, s);
        g.ws = ws + pl.dp + pl.sums;
        g.ws_bytes = static_cast<size_t>(pl.gemm);
        e = gemm_run(g, dev, &launches);
    };
    run(DGA_ROW_MAJOR, M, 2 * F, W, ldw, dX, lddx);
    run(DGA_COL_MAJOR, 2 * F, M, X, ldx, dW, lddw);
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

int dga_q4_quantize(dga_dtype in_dtype, dga_dtype scale_dtype, int64_t rows, int64_t cols, int group, const void* W, int64_t ldw,
                    void* codes, int64_t ld_codes, void* scales, int64_t ld_scales, void* zeros, int64_t ld_zeros,
                    dga_stream_t stream) {
    if (!float_type(in_dtype) || !half_type(scale_dtype) || !group_ok(group)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(rows)) return -3;
    if (!dim_ok(cols)) return -4;
    set_last_launches(0);
    if (rows == 0 || cols == 0) return DGA_OK;
    const int64_t es = type_size(in_dtype);
    if (!W || !aligned(W, es)) return -6;
    if (ldw < cols) return -7;
    const Q4Matrix q{static_cast<uint8_t*>(codes), ld_codes, scales, ld_scales, static_cast<uint8_t*>(zeros), ld_zeros, group};
    const int bad = check_q4(q, cols, 8);
    if (bad) return -bad;
    Arrays a;
    a.in(W, rows, ldw * es, cols * es);
    q4_arrays(a, q, rows, cols, true);
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    const cudaError_t e = q4_quantize_launch(in_dtype, scale_dtype, rows, cols, W, ldw, q, dev, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(1);
    return DGA_OK;
}

int dga_q4_dequantize(dga_dtype scale_dtype, dga_dtype out_dtype, int64_t rows, int64_t cols, int group, const void* codes,
                      int64_t ld_codes, const void* scales, int64_t ld_scales, const void* zeros, int64_t ld_zeros, void* Y,
                      int64_t ldy, dga_stream_t stream) {
    if (!half_type(scale_dtype) || !float_type(out_dtype) || !group_ok(group)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(rows)) return -3;
    if (!dim_ok(cols)) return -4;
    set_last_launches(0);
    if (rows == 0 || cols == 0) return DGA_OK;
    const Q4Matrix q{static_cast<const uint8_t*>(codes), ld_codes, scales, ld_scales, static_cast<const uint8_t*>(zeros), ld_zeros, group};
    const int bad = check_q4(q, cols, 6);
    if (bad) return -bad;
    const int64_t es = type_size(out_dtype);
    if (!Y || !aligned(Y, es)) return -12;
    if (ldy < cols) return -13;
    Arrays a;
    q4_arrays(a, q, rows, cols, false);
    a.out(Y, rows, ldy * es, cols * es);
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    const cudaError_t e = q4_dequantize_launch(scale_dtype, out_dtype, rows, cols, q, Y, ldy, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(1);
    return DGA_OK;
}

size_t dga_q4_linear_workspace_size(dga_dtype dtype, int64_t M, int64_t N, int64_t K, int64_t ldx) {
    if (!half_type(dtype) || M <= 0 || N <= 0 || !dim_ok(M) || !dim_ok(N) || !dim_ok(K)) return 0;
    return static_cast<size_t>(q4_plan(dtype, M, N, K, ldx, false, nullptr).total());
}

int dga_q4_linear(dga_dtype dtype, int64_t M, int64_t N, int64_t K, int group, const void* X, int64_t ldx, const void* codes,
                  int64_t ld_codes, const void* scales, int64_t ld_scales, const void* zeros, int64_t ld_zeros, const void* bias,
                  void* Y, int64_t ldy, void* workspace, size_t workspace_bytes, dga_stream_t stream) {
    if (!half_type(dtype) || !group_ok(group)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(M)) return -2;
    if (!dim_ok(N)) return -3;
    if (!dim_ok(K)) return -4;
    set_last_launches(0);
    if (M == 0 || N == 0) return DGA_OK;
    if (K > 0 && (!X || !aligned(X, 2))) return -6;
    if (ldx < at_least_one(K)) return -7;
    const Q4Matrix q{static_cast<const uint8_t*>(codes), ld_codes, scales, ld_scales, static_cast<const uint8_t*>(zeros), ld_zeros, group};
    const int bad = K > 0 ? check_q4(q, K, 8) : 0;
    if (bad) return -bad;
    if (bias && !aligned(bias, 2)) return -14;
    if (!Y || !aligned(Y, 2)) return -15;
    if (ldy < N) return -16;
    if ((workspace_bytes > 0 && !workspace) || (workspace && !aligned(workspace, 256))) return -17;
    const Q4Plan pl = q4_plan(dtype, M, N, K, ldx, false, X);
    if (workspace_bytes < static_cast<size_t>(pl.total())) return DGA_ERR_WORKSPACE;
    Arrays a;
    if (K > 0) a.in(X, M, ldx * 2, K * 2), q4_arrays(a, q, N, K, false);
    a.in(bias, 1, 0, N * 2);
    a.out(Y, M, ldy * 2, N * 2);
    a.out(workspace, 1, 0, pl.total());
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int launches = 0;
    cudaError_t e;
    if (pl.rows || pl.tensor) {
        e = q4_by_kernel(pl, dtype, 0, M, N, K, X, ldx, q, bias, Y, ldy, false, static_cast<uint8_t*>(workspace), dev, s, &launches);
    } else {
        e = q4_by_values(pl, dtype, dtype, M, N, K, X, ldx, q, bias, Y, ldy, static_cast<uint8_t*>(workspace), dev, s, &launches);
    }
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

size_t dga_q4_gated_workspace_size(dga_dtype dtype, int64_t M, int64_t F, int64_t K, int64_t ldx) {
    if (!half_type(dtype) || M <= 0 || F <= 0 || !dim_ok(M) || !dim_ok(F) || !dim_ok(K)) return 0;
    return static_cast<size_t>(q4_plan(dtype, M, 2 * F, K, ldx, true, nullptr).total());
}

int dga_q4_gated(dga_dtype dtype, dga_activation act, int64_t M, int64_t F, int64_t K, int group, const void* X, int64_t ldx,
                 const void* codes, int64_t ld_codes, const void* scales, int64_t ld_scales, const void* zeros, int64_t ld_zeros,
                 const void* bias, void* H, int64_t ldh, void* workspace, size_t workspace_bytes, dga_stream_t stream) {
    if (!half_type(dtype) || !act_ok(act) || !group_ok(group)) return DGA_ERR_UNSUPPORTED;
    if (!dim_ok(M)) return -3;
    if (!dim_ok(F)) return -4;
    if (!dim_ok(K)) return -5;
    set_last_launches(0);
    if (M == 0 || F == 0) return DGA_OK;
    if (K > 0 && (!X || !aligned(X, 2))) return -7;
    if (ldx < at_least_one(K)) return -8;
    const Q4Matrix q{static_cast<const uint8_t*>(codes), ld_codes, scales, ld_scales, static_cast<const uint8_t*>(zeros), ld_zeros, group};
    const int bad = K > 0 ? check_q4(q, K, 9) : 0;
    if (bad) return -bad;
    if (bias && !aligned(bias, 2)) return -15;
    if (!H || !aligned(H, 2)) return -16;
    if (ldh < F) return -17;
    if ((workspace_bytes > 0 && !workspace) || (workspace && !aligned(workspace, 256))) return -18;
    const Q4Plan pl = q4_plan(dtype, M, 2 * F, K, ldx, true, X);
    if (workspace_bytes < static_cast<size_t>(pl.total())) return DGA_ERR_WORKSPACE;
    Arrays a;
    if (K > 0) a.in(X, M, ldx * 2, K * 2), q4_arrays(a, q, 2 * F, K, false);
    a.in(bias, 1, 0, 2 * F * 2);
    a.out(H, M, ldh * 2, F * 2);
    a.out(workspace, 1, 0, pl.total());
    if (a.meet()) return DGA_ERR_OVERLAP;
    DeviceInfo dev;
    const int st = device(&dev);
    if (st != DGA_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int launches = 0;
    cudaError_t e;
    if (K > 0) {
        e = q4_by_kernel(pl, dtype, act, M, F, K, X, ldx, q, bias, H, ldh, true, ws, dev, s, &launches);
    } else {
        e = q4_by_values(pl, dtype, DGA_F32, M, 2 * F, K, X, ldx, q, nullptr, ws + pl.values, held_ld(F), ws, dev, s, &launches);
        if (e != cudaSuccess) return note_cuda_error(e);
        e = gated_act_launch(dtype, act, M, F, reinterpret_cast<const float*>(ws + pl.values), held_ld(F), bias, H, ldh, nullptr, 0, s);
        if (e == cudaSuccess) ++launches;
    }
    if (e != cudaSuccess) return note_cuda_error(e);
    set_last_launches(launches);
    return DGA_OK;
}

}  // extern "C"
