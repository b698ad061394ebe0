// q4_rows.cu -- products of a few rows with a 4-bit weight with group scales,
//     Y[M, N] = X[M, K] ((q - z) s)[N, K]^T + bias,    M <= 64,
// and the gated layer H = act(g) * u on them.
//
// The bytes of the codes bound it (half a byte to a weight), so each is read
// once, straight into registers, and is multiplied as what it is: q - z is a
// small integer, exact in bf16 and fp16, and mma.sync m16n8k16 multiplies it by
// X exactly and sums a group in fp32; the group's sum is then scaled by s in
// fp32.  No weight is rounded.
//
//  * A block of 8 warps takes kTiles tiles of 16 weight rows (of a gated layer
//    half of them gate rows and half the up rows that go with them) and all of
//    K, its warps every eighth run of 128 columns; their sums are added through
//    shared memory in a fixed order, and the activation and the product of a
//    gated layer follow from there.
//  * The weight is the MMA's A (16 rows), X its B (8 rows).  Which k an MMA's
//    columns stand for is free as long as A and B agree, so a lane reads
//    consecutive codes of its two rows: in a run of 128, groups of 128 give a lane
//    16 bytes, groups of 64 twice 8 bytes, groups of 32 four times 4 bytes, so
//    that an MMA's columns are of one group.
//  * A word of 8 codes becomes four registers of two: (w >> 4 i) & 0x000f000f
//    has codes i and i + 4, and or-ed into the mantissa of 128 (bf16) or 1024
//    (fp16) they are 128 + q or 1024 + q; subtracting 128 + z or 1024 + z is
//    exact.  X's eight values are paired alike.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "gated_act.cuh"
#include "mx_common.cuh"

namespace dga {
namespace {

constexpr int kWarps = 8;
constexpr int kRun = 128;  // columns a warp takes at a time

struct RowsParams {
    int64_t M, N, K;  // N: outputs (a gated layer's F)
    const void* X;
    int64_t ldx;
    Q4Matrix q;
    const void* bias;
    void* Y;
    int64_t ldy;
    int act;
    int x_vec;      // X's rows take 16-byte loads
    int scale_vec;  // a run's scales (zero points) are one aligned word
};

template <typename T> struct Codes;
template <> struct Codes<__nv_bfloat16> {
    static constexpr uint32_t kBase = 0x43004300u;  // 128, 128
    __device__ __forceinline__ static uint32_t minus(uint32_t a, uint32_t b) {
        __nv_bfloat162 x, y;
        memcpy(&x, &a, 4);
        memcpy(&y, &b, 4);
        x = __hsub2(x, y);
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ __forceinline__ static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
template <> struct Codes<__half> {
    static constexpr uint32_t kBase = 0x64006400u;  // 1024, 1024
    __device__ __forceinline__ static uint32_t minus(uint32_t a, uint32_t b) {
        __half2 x, y;
        memcpy(&x, &a, 4);
        memcpy(&y, &b, 4);
        x = __hsub2(x, y);
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ __forceinline__ static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// The four words of codes that lane t of a quad has of a run of a row.
template <int kGroup>
__device__ __forceinline__ void load_codes(uint32_t (&w)[4], const uint8_t* run, int t, int bytes_left) {
    if constexpr (kGroup == 128) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t * 16 < bytes_left) v = __ldg(reinterpret_cast<const uint4*>(run + t * 16));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kGroup == 64) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint2 v = make_uint2(0, 0);
            if (h * 32 + t * 8 < bytes_left) v = __ldg(reinterpret_cast<const uint2*>(run + h * 32 + t * 8));
            w[2 * h] = v.x, w[2 * h + 1] = v.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = j * 16 < bytes_left ? __ldg(reinterpret_cast<const uint32_t*>(run + j * 16 + t * 4)) : 0u;
    }
}
// The column, within the run, of the first of word j's codes.
template <int kGroup>
__device__ __forceinline__ int word_column(int j, int t) {
    if constexpr (kGroup == 128) return t * 32 + j * 8;
    else if constexpr (kGroup == 64) return (j >> 1) * 64 + t * 16 + (j & 1) * 8;
    else return j * 32 + t * 8;
}

// Eight values of a row of X from column k on, zero past K, paired as the codes are.
template <typename T>
__device__ __forceinline__ void load_x(uint32_t (&b)[4], const T* row, int64_t k, int64_t K, int vec) {
    uint32_t v[4];
    if (vec && k + 8 <= K) {
        const uint4 r = __ldg(reinterpret_cast<const uint4*>(row + k));
        v[0] = r.x, v[1] = r.y, v[2] = r.z, v[3] = r.w;
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = k + 2 * i < K ? __ldg(p + k + 2 * i) : 0u, hi = k + 2 * i + 1 < K ? __ldg(p + k + 2 * i + 1) : 0u;
            v[i] = lo | (hi << 16);
        }
    }
    b[0] = __byte_perm(v[0], v[2], 0x5410);  // values 0 and 4
    b[1] = __byte_perm(v[0], v[2], 0x7632);  // 1 and 5
    b[2] = __byte_perm(v[1], v[3], 0x5410);  // 2 and 6
    b[3] = __byte_perm(v[1], v[3], 0x7632);  // 3 and 7
}

// A run's scales (as fp32) and bases (128 or 1024 plus the zero point, twice) of a row;
// groups past the row's last give 0.
template <typename T, int kGroup>
__device__ __forceinline__ void load_scales(float (&s)[kRun / kGroup], uint32_t (&z)[kRun / kGroup], const Q4Matrix& q, int64_t row,
                                            int64_t group, int64_t groups, int vec) {
    constexpr int kN = kRun / kGroup;
    const T* sp = static_cast<const T*>(q.scales) + row * q.ld_scales + group;
    const uint8_t* zp = q.zeros ? q.zeros + row * q.ld_zeros + group : nullptr;
    T t[kN];
    uint32_t zero = 0x08080808u;
    if (vec && group + kN <= groups) {
        if constexpr (kN == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(sp));
            memcpy(t, &v, 8);
            if (zp) zero = __ldg(reinterpret_cast<const uint32_t*>(zp));
        } else if constexpr (kN == 2) {
            const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(sp));
            memcpy(t, &v, 4);
            if (zp) zero = __ldg(reinterpret_cast<const uint16_t*>(zp));
        } else {
            t[0] = *sp;
            if (zp) zero = __ldg(zp);
        }
    } else {
        if (zp) zero = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const bool in = group + i < groups;
            t[i] = in ? sp[i] : T(0.0f);
            if (zp && in) zero |= static_cast<uint32_t>(__ldg(zp + i)) << (8 * i);
        }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        s[i] = static_cast<float>(t[i]);
        z[i] = Codes<T>::kBase | (((zero >> (8 * i)) & 15u) * 0x00010001u);
    }
}

// kTiles: tiles of 16 weight rows to a block; kMt: tiles of 8 rows of X.
template <typename T, int kGroup, int kMt, int kTiles, bool kGated>
__global__ void __launch_bounds__(kWarps * 32) q4_rows_kernel(RowsParams p) {
    static_assert(!kGated || kTiles % 2 == 0, "as many up tiles as gate tiles");
    constexpr int kRows = kTiles * 16, kOut = kGated ? kRows / 2 : kRows, kPitch = kRows + 4;
    extern __shared__ float part[];  // [warp][8 kMt][kPitch]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kOut;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the weight rows of this lane: g and g + 8 of each tile (past the last, the last)
    int64_t rows[kTiles][2];
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = (r * 16 + h * 8 + g) % kOut;
            rows[r][h] = min(n0 + at, p.N - 1) + (r * 16 >= kOut ? p.N : 0);
        }
    float acc[kTiles][kMt][4];
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][m][i] = 0.0f;

    const T* X = static_cast<const T*>(p.X);
    const int64_t row_bytes = mx_row_bytes(p.K), groups = (p.K + kGroup - 1) / kGroup;
    const int64_t runs = (p.K + kRun - 1) / kRun;
    for (int64_t run = warp; run < runs; run += kWarps) {
        const int left = static_cast<int>(min(static_cast<int64_t>(64), row_bytes - run * 64));
        uint32_t w[kTiles][2][4];
#pragma unroll
        for (int r = 0; r < kTiles; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) load_codes<kGroup>(w[r][h], p.q.codes + rows[r][h] * p.q.ld + run * 64, t, left);
        float s[kTiles][2][kRun / kGroup];
        uint32_t z[kTiles][2][kRun / kGroup];
#pragma unroll
        for (int r = 0; r < kTiles; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                load_scales<T, kGroup>(s[r][h], z[r][h], p.q, rows[r][h], run * (kRun / kGroup), groups, p.scale_vec);
        float sum[kTiles][kMt][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            constexpr int kWords = kGroup / 32;  // words of a lane to a group
            const int64_t k = run * kRun + word_column<kGroup>(j, t);
            uint32_t b[kMt][4];
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
                const int64_t row = m * 8 + g;
                if (row < p.M) load_x(b[m], X + row * p.ldx, k, p.K, p.x_vec);
                else b[m][0] = b[m][1] = b[m][2] = b[m][3] = 0;
            }
#pragma unroll
            for (int r = 0; r < kTiles; ++r) {
                if (j % kWords == 0) {
#pragma unroll
                    for (int m = 0; m < kMt; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[r][m][i] = 0.0f;
                }
                uint32_t c[4][2];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        c[i][h] = Codes<T>::minus(((w[r][h][j] >> (4 * i)) & 0x000f000fu) | Codes<T>::kBase, z[r][h][j / kWords]);
                const uint32_t a0[4] = {c[0][0], c[0][1], c[1][0], c[1][1]}, a1[4] = {c[2][0], c[2][1], c[3][0], c[3][1]};
#pragma unroll
                for (int m = 0; m < kMt; ++m) {
                    Codes<T>::mma(sum[r][m], a0, b[m][0], b[m][1]);
                    Codes<T>::mma(sum[r][m], a1, b[m][2], b[m][3]);
                }
                if (j % kWords == kWords - 1) {
#pragma unroll
                    for (int m = 0; m < kMt; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[r][m][i] = fmaf(s[r][i >> 1][j / kWords], sum[r][m][i], acc[r][m][i]);
                }
            }
        }
    }

    // sum[..][2h + i]: weight row g + 8h of the tile, row 2t + i of X's tile
    float* mine = part + warp * (8 * kMt * kPitch);
#pragma unroll
    for (int r = 0; r < kTiles; ++r)
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                mine[(m * 8 + 2 * t + (i & 1)) * kPitch + r * 16 + g + 8 * (i >> 1)] = acc[r][m][i];
    __syncthreads();
    const T* bias = static_cast<const T*>(p.bias);
    for (int o = threadIdx.x; o < 8 * kMt * kOut; o += kWarps * 32) {
        const int row = o / kOut, c = o % kOut;
        const int64_t n = n0 + c;
        if (row >= p.M || n >= p.N) continue;
        auto total = [&](int col) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v += part[(k * 8 * kMt + row) * kPitch + col];
            return v;
        };
        float v = total(c);
        if (bias) v += OutT<T>::load(bias + n);
        if constexpr (kGated) {
            float u = total(kOut + c);
            if (bias) u += OutT<T>::load(bias + p.N + n);
            switch (p.act) {
            case DGA_SILU: v = act_value<DGA_SILU, true>(v); break;
            case DGA_GELU: v = act_value<DGA_GELU, true>(v); break;
            case DGA_GELU_TANH: v = act_value<DGA_GELU_TANH, true>(v); break;
            case DGA_RELU: v = act_value<DGA_RELU, true>(v); break;
            default: v = act_value<DGA_SIGMOID, true>(v); break;
            }
            v *= u;
        }
        OutT<T>::store(static_cast<T*>(p.Y) + row * p.ldy + n, v);
    }
}

template <typename T, int kGroup, int kMt, int kTiles, bool kGated>
cudaError_t launch(const RowsParams& p, cudaStream_t s) {
    constexpr int kOut = kGated ? kTiles * 8 : kTiles * 16;
    constexpr int kSmem = kWarps * 8 * kMt * (kTiles * 16 + 4) * 4;
    auto kern = q4_rows_kernel<T, kGroup, kMt, kTiles, kGated>;
    if (kSmem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + kOut - 1) / kOut));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T, int kGroup>
cudaError_t launch_rows(const RowsParams& p, bool gated, cudaStream_t s) {
    if (gated) {
        if (p.M <= 8) return launch<T, kGroup, 1, 2, true>(p, s);
        if (p.M <= 16) return launch<T, kGroup, 2, 2, true>(p, s);
        if (p.M <= 32) return launch<T, kGroup, 4, 2, true>(p, s);
        return launch<T, kGroup, 8, 2, true>(p, s);
    }
    if (p.M <= 8) return launch<T, kGroup, 1, 1, false>(p, s);
    if (p.M <= 16) return launch<T, kGroup, 2, 2, false>(p, s);
    if (p.M <= 32) return launch<T, kGroup, 4, 2, false>(p, s);
    return launch<T, kGroup, 8, 2, false>(p, s);
}

template <typename T>
cudaError_t launch_group(const RowsParams& p, bool gated, cudaStream_t s) {
    return p.q.group == 32 ? launch_rows<T, 32>(p, gated, s)
           : p.q.group == 64 ? launch_rows<T, 64>(p, gated, s) : launch_rows<T, 128>(p, gated, s);
}

}  // namespace

cudaError_t q4_rows_launch(int dtype, int act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const Q4Matrix& q,
                           const void* bias, void* Y, int64_t ldy, bool gated, cudaStream_t stream) {
    RowsParams p{};
    p.M = M, p.N = N, p.K = K;
    p.X = X, p.ldx = ldx;
    p.q = q;
    p.bias = bias;
    p.Y = Y, p.ldy = ldy;
    p.act = act;
    p.x_vec = aligned(X, 16) && ldx % 8 == 0;
    const int64_t n = kRun / q.group;
    p.scale_vec = aligned(q.scales, 2 * n) && q.ld_scales % n == 0 && (!q.zeros || (aligned(q.zeros, n) && q.ld_zeros % n == 0));
    return dtype == DGA_BF16 ? launch_group<__nv_bfloat16>(p, gated, stream) : launch_group<__half>(p, gated, stream);
}

}  // namespace dga
