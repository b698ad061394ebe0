// gated.cu -- the element-wise passes of the gated feed-forward layer
//     P = X W^T + b = [g | u],  H = act(g) * u
// around the library's GEMM: the activation and the product of pre-activations
// that a GEMM wrote, and their gradient
//     dP = [G u act'(g) | G act(g)]
// with the bias's gradient, dP's column sums, from the same pass.  Bound by
// memory: every value is read and written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dga_internal.h"
#include "gated_act.cuh"

namespace dga {
namespace {

// ---- H (and P in its type) from pre-activations ------------------------------------
//
// A thread kVec values of a row; the grid's y walks the rows.
template <typename T, int kAct, int kVec>
__global__ void __launch_bounds__(256)
    act_kernel(int64_t M, int64_t F, const float* __restrict__ P, int64_t ldp, const T* __restrict__ bias, T* __restrict__ H,
               int64_t ldh, T* __restrict__ Pout, int64_t ld_out) {
    constexpr bool kFast = sizeof(T) == 2;
    const int64_t f = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * kVec;
    if (f >= F) return;
    float bg[kVec], bu[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        bg[i] = bias != nullptr ? static_cast<float>(bias[f + i]) : 0.0f;
        bu[i] = bias != nullptr ? static_cast<float>(bias[F + f + i]) : 0.0f;
    }
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        float g[kVec], u[kVec], h[kVec];
        Pack<float, kVec>::load(P + m * ldp + f, g);
        Pack<float, kVec>::load(P + m * ldp + F + f, u);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            g[i] += bg[i];
            u[i] += bu[i];
            h[i] = act_value<kAct, kFast>(g[i]) * u[i];
        }
        Pack<T, kVec>::store(H + m * ldh + f, h);
        if (Pout != nullptr) {
            Pack<T, kVec>::store(Pout + m * ld_out + f, g);
            Pack<T, kVec>::store(Pout + m * ld_out + F + f, u);
        }
    }
}

// ---- dP and its column sums ----------------------------------------------------------
//
// A block takes 32 * kVec columns of G and a slice of the rows, its 8 warps
// every eighth row of it with kRows rows in flight.  The sums of a slice go to
// partials[slice][2F] in a fixed order, and sum_slices_kernel adds the slices.
constexpr int kGradWarps = 8;

template <typename T, int kAct, int kVec>
__global__ void __launch_bounds__(kGradWarps * 32)
    grad_kernel(int64_t M, int64_t F, const T* __restrict__ P, int64_t ldp, const T* __restrict__ G, int64_t ldg,
                T* __restrict__ dP, int64_t ldd, float* __restrict__ partials) {
    constexpr bool kFast = sizeof(T) == 2;
    constexpr int kRows = 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t f = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * kVec;
    const int64_t per = (M + gridDim.y - 1) / gridDim.y;
    const int64_t begin = min(M, blockIdx.y * per), end = min(M, begin + per);
    float sg[kVec], su[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) sg[i] = su[i] = 0.0f;
    if (f < F) {
        auto one = [&](int64_t m, const float (&g)[kVec], const float (&u)[kVec], const float (&d)[kVec]) {
            float dg[kVec], du[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                float value, slope;
                act_both<kAct, kFast>(g[i], value, slope);
                dg[i] = d[i] * u[i] * slope;
                du[i] = d[i] * value;
                sg[i] += dg[i];
                su[i] += du[i];
            }
            Pack<T, kVec>::store(dP + m * ldd + f, dg);
            Pack<T, kVec>::store(dP + m * ldd + F + f, du);
        };
        int64_t m = begin + warp;
        for (; m + (kRows - 1) * kGradWarps < end; m += kRows * kGradWarps) {
            float g[kRows][kVec], u[kRows][kVec], d[kRows][kVec];
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int64_t at = m + r * kGradWarps;
                Pack<T, kVec>::load(P + at * ldp + f, g[r]);
                Pack<T, kVec>::load(P + at * ldp + F + f, u[r]);
                Pack<T, kVec>::load(G + at * ldg + f, d[r]);
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) one(m + r * kGradWarps, g[r], u[r], d[r]);
        }
        for (; m < end; m += kGradWarps) {
            float g[kVec], u[kVec], d[kVec];
            Pack<T, kVec>::load(P + m * ldp + f, g);
            Pack<T, kVec>::load(P + m * ldp + F + f, u);
            Pack<T, kVec>::load(G + m * ldg + f, d);
            one(m, g, u, d);
        }
    }
    if (partials == nullptr) return;
    __shared__ float part[kGradWarps][2][32 * kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        part[warp][0][lane * kVec + i] = sg[i];
        part[warp][1][lane * kVec + i] = su[i];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 64 * kVec; c += kGradWarps * 32) {
        const int half = c / (32 * kVec), j = c % (32 * kVec);
        const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * kVec + j;
        if (col >= F) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kGradWarps; ++w) s += part[w][half][j];
        partials[blockIdx.y * 2 * F + half * F + col] = s;
    }
}

__global__ void __launch_bounds__(256) sum_slices_kernel(int64_t cols, int slices, const float* __restrict__ partials,
                                                         float* __restrict__ out) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (c >= cols) return;
    float s = 0.0f;
#pragma unroll 8
    for (int i = 0; i < slices; ++i) s += partials[i * cols + c];
    out[c] = s;
}

// ---- rows of 16-bit values to rows that start on 16 bytes -------------------------------
//
// Eight values of a row to a thread, four rows of them in flight; zero past the
// row's end; read by words of two, and shifted where the row starts between two (at
// the array's ends one by one).  The grid's z is the array: a call's two in one
// launch (a gated layer of 300 x 2051 to 700, whose X and W both need it: 27.5 us a
// call from the host, some 4 more with two launches; 23.4 us in a graph).
constexpr int kCopyX = 64, kCopyY = 4, kCopyRows = 4;

__global__ void __launch_bounds__(kCopyX * kCopyY) copy_rows_kernel(CopyRows a, CopyRows b) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const CopyRows& c = blockIdx.z == 0 ? a : b;
    const int64_t k = (static_cast<int64_t>(blockIdx.x) * kCopyX + threadIdx.x) * 8;
    if (k >= c.ldy) return;
    const uint16_t* X = static_cast<const uint16_t*>(c.X);
    for (int64_t row0 = (static_cast<int64_t>(blockIdx.y) * kCopyY + threadIdx.y) * kCopyRows; row0 < c.rows;
         row0 += static_cast<int64_t>(gridDim.y) * kCopyY * kCopyRows) {
        uint32_t w[kCopyRows][5];
#pragma unroll
        for (int r = 0; r < kCopyRows; ++r) {
            const int64_t row = min(row0 + r, c.rows - 1);
            const uint16_t* src = X + row * c.ldx + k;
#pragma unroll
            for (int j = 0; j < 5; ++j) w[r][j] = 0;
            if (k + 8 < c.cols && (row > 0 || k > 0)) {
                const uint32_t odd = (reinterpret_cast<uintptr_t>(src) >> 1) & 1;
                const uint32_t* words = reinterpret_cast<const uint32_t*>(src - odd);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[r][j] = __ldg(words + j);
                if (odd) w[r][4] = __ldg(words + 4);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k + j < c.cols) w[r][j / 2] |= static_cast<uint32_t>(__ldg(src + j)) << (16 * (j & 1));
            }
        }
#pragma unroll
        for (int r = 0; r < kCopyRows; ++r) {
            const int64_t row = row0 + r;
            if (row >= c.rows) break;
            const uint16_t* src = X + row * c.ldx + k;
            if (k + 8 < c.cols && (row > 0 || k > 0) && ((reinterpret_cast<uintptr_t>(src) >> 1) & 1)) {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[r][j] = __funnelshift_r(w[r][j], w[r][j + 1], 16);
            }
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(c.Y) + row * c.ldy + k) = make_uint4(w[r][0], w[r][1], w[r][2], w[r][3]);
        }
    }
}

// Row slices of the gradient pass: about 16 blocks to an SM at 256 columns to
// a block, none under 32 rows.
int grad_slices(int64_t M, int64_t F) {
    const int64_t tiles = std::max<int64_t>(1, (F + 255) / 256);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(M + 31) / 32, std::max<int64_t>(16, 2432 / tiles), 256})));
}

template <typename Fn>
cudaError_t for_act(int act, Fn&& f) {
    switch (act) {
    case DGA_SILU: return f(std::integral_constant<int, DGA_SILU>{});
    case DGA_GELU: return f(std::integral_constant<int, DGA_GELU>{});
    case DGA_GELU_TANH: return f(std::integral_constant<int, DGA_GELU_TANH>{});
    case DGA_RELU: return f(std::integral_constant<int, DGA_RELU>{});
    case DGA_SIGMOID: return f(std::integral_constant<int, DGA_SIGMOID>{});
    default: return cudaErrorInvalidValue;
    }
}

template <typename Fn>
cudaError_t for_type(int dtype, Fn&& f) {
    switch (dtype) {
    case DGA_F32: return f(float{});
    case DGA_BF16: return f(__nv_bfloat16{});
    case DGA_F16: return f(__half{});
    default: return cudaErrorInvalidValue;
    }
}

// Whether rows of this leading dimension can be read kVec values at a time.
bool vectors(const void* p, int64_t ld, int vec, int64_t size) {
    return aligned(p, static_cast<size_t>(vec * size)) && ld % vec == 0;
}

}  // namespace

cudaError_t copy_rows_launch(const CopyRows& a, const CopyRows* b, cudaStream_t stream) {
    const int64_t ld = std::max(a.ldy, b ? b->ldy : 0), rows = std::max(a.rows, b ? b->rows : 0);
    const int64_t per = kCopyY * kCopyRows;
    const dim3 grid(static_cast<unsigned>((ld + kCopyX * 8 - 1) / (kCopyX * 8)),
                    static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, 65535)), b ? 2 : 1);
    copy_rows_kernel<<<grid, dim3(kCopyX, kCopyY), 0, stream>>>(a, b ? *b : a);
    return cudaGetLastError();
}

cudaError_t gated_act_launch(int dtype, int act, int64_t M, int64_t F, const float* P, int64_t ldp, const void* bias, void* H,
                             int64_t ldh, void* Pout, int64_t ld_out, cudaStream_t stream) {
    const int64_t es = dtype == DGA_F32 ? 4 : 2;
    const bool vec = F % 4 == 0 && vectors(P, ldp, 4, 4) && vectors(H, ldh, 4, es) &&
                     (Pout == nullptr || vectors(Pout, ld_out, 4, es));
    const int64_t x = (F + (vec ? 1023 : 255)) / (vec ? 1024 : 256);
    if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(std::min<int64_t>(M, 65535)));
    return for_type(dtype, [&](auto t) {
        return for_act(act, [&](auto a) {
            using T = decltype(t);
            auto kern = vec ? act_kernel<T, decltype(a)::value, 4> : act_kernel<T, decltype(a)::value, 1>;
            kern<<<grid, 256, 0, stream>>>(M, F, P, ldp, static_cast<const T*>(bias), static_cast<T*>(H), ldh,
                                           static_cast<T*>(Pout), ld_out);
            return cudaGetLastError();
        });
    });
}

size_t gated_grad_partials(int64_t M, int64_t F) { return static_cast<size_t>(grad_slices(M, F)) * 2 * F; }

cudaError_t gated_grad_launch(int dtype, int act, int64_t M, int64_t F, const void* P, int64_t ldp, const void* G,
                              int64_t ldg, void* dP, int64_t ldd, float* db, float* partials, cudaStream_t stream,
                              int* launches) {
    const int slices = grad_slices(M, F);
    cudaError_t e = for_type(dtype, [&](auto t) {
        return for_act(act, [&](auto a) {
            using T = decltype(t);
            constexpr int kVec = 16 / sizeof(T);
            const bool vec = F % kVec == 0 && vectors(P, ldp, kVec, sizeof(T)) && vectors(G, ldg, kVec, sizeof(T)) &&
                             vectors(dP, ldd, kVec, sizeof(T));
            const int64_t cols = vec ? 32 * kVec : 32;
            const int64_t x = (F + cols - 1) / cols;
            if (x > 0x7fffffff) return cudaErrorInvalidConfiguration;
            auto kern = vec ? grad_kernel<T, decltype(a)::value, kVec> : grad_kernel<T, decltype(a)::value, 1>;
            kern<<<dim3(static_cast<unsigned>(x), slices), kGradWarps * 32, 0, stream>>>(
                M, F, static_cast<const T*>(P), ldp, static_cast<const T*>(G), ldg, static_cast<T*>(dP), ldd,
                db ? partials : nullptr);
            return cudaGetLastError();
        });
    });
    if (e != cudaSuccess) return e;
    ++*launches;
    if (db == nullptr) return cudaSuccess;
    sum_slices_kernel<<<static_cast<unsigned>((2 * F + 255) / 256), 256, 0, stream>>>(2 * F, slices, partials, db);
    e = cudaGetLastError();
    if (e == cudaSuccess) ++*launches;
    return e;
}

}  // namespace dga
