// mx_quant.cu -- a matrix to 4-bit microscaled form and back.
//
// For each block of 32 (MXFP4) or 16 (NVFP4) consecutive values of a row,
// with m = max |x| over the block:
//   MXFP4  scale 2^e, e = floor(log2 m) - 2 held to [-127, 127] (2 being the
//          exponent of E2M1's largest value): the MX specification's rule
//   NVFP4  scale s = E4M3(min(448, m / (6 g))), g the tensor's factor (1 if
//          there is none), rounded to nearest even; the unit is s g
//   code   E2M1(x / unit), nearest even, magnitudes over 6 becoming 6
// A block with an infinity or a NaN gets a NaN scale, so that it reads back
// as NaN; an all-zero block gets the smallest scale.
//
// Every step is exact or correctly rounded in fp32, so the codes and scales
// are those of the definition, whatever the order of the work: 2^-e is a
// power of two; x / unit is the correctly rounded quotient.
//
// Bound by memory: 2 or 4 bytes read and 0.53 or 0.56 written per value.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "dga_internal.h"
#include "mx_common.cuh"
#include "mx_quant.cuh"

namespace dga {
namespace {

// Eight codes to their values.
__device__ __forceinline__ void values8(uint32_t c, float (&v)[8]) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(c));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        v[2 * q] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[q] & 0xffff)));
        v[2 * q + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(h[q] >> 16)));
    }
}

// Eight consecutive values of a row, zero past its end.  `vec`: the row's
// groups of four are 16-byte aligned.
__device__ __forceinline__ void load8(const float* __restrict__ row, int64_t k, int64_t K, bool vec, float (&x)[8]) {
    if (vec && k + 8 <= K) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(row + k)), b = __ldg(reinterpret_cast<const float4*>(row + k) + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = k + q < K ? row[k + q] : 0.0f;
    }
}

// These kernels are launched as programmatic dependents: their blocks may be
// placed while the kernel before still runs, and wait here for its end.  Then a
// product launched behind this one may be placed: it reads its weight at once,
// which was complete before this grid's start, and waits for this grid's end
// before it reads what is written here.  (The gradients of a 4096 x 4096 layer for 4096
// tokens: 122 to 109 us.)
__device__ __forceinline__ void begin_after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- along rows ------------------------------------------------------------
//
// 16-bit sources: a thread takes 32 consecutive values of a row, one block
// (MXFP4) or two (NVFP4): four 16-byte loads, maxima of packed magnitudes, one
// 16-byte store of codes and its scale byte(s).  Nothing is shared between
// lanes and nothing computed twice; with eight values to a lane and a block's
// maximum and scale found by 2 or 4 lanes it was bound by instructions (8192 x
// 8192 bf16: 51 us MXFP4, 70 us NVFP4).
// Rows that do not start on 16 bytes are read by the aligned pieces that cover
// them, shifted in registers (4093 x 4099 bf16, MXFP4:
// 16 us, element by element 35 us).
// fp32 sources: eight values to a lane as just described, since 128 bytes to a
// lane would be bound by the L1's lines (8192 x 8192: 49 us MXFP4, 64 us NVFP4).

// 16 words from `src`, an address of 16-bit values: the five aligned 16-byte
// pieces around them, shifted by 8, 4 and 2 bytes as the address asks.
__device__ __forceinline__ void load_words_shifted(const void* src, uint32_t (&w)[16]) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(src)) & 15;
    const uint4* at = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(src) - off);
    uint32_t x[20];
#pragma unroll
    for (int q = 0; q < 5; ++q) {
        const uint4 v = __ldg(at + q);
        x[4 * q] = v.x, x[4 * q + 1] = v.y, x[4 * q + 2] = v.z, x[4 * q + 3] = v.w;
    }
#pragma unroll
    for (int j = 0; j < 18; ++j) x[j] = off & 8 ? x[j + 2] : x[j];
#pragma unroll
    for (int j = 0; j < 17; ++j) x[j] = off & 4 ? x[j + 1] : x[j];
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = __funnelshift_r(x[j], x[j + 1], (off & 2) * 8);
}

template <int kFormat, typename T>
__global__ void __launch_bounds__(256) mx_quant_rows16_kernel(const T* __restrict__ X, int64_t ldx, uint32_t rows, int64_t K,
                                                              bool vec, const float* __restrict__ factor,
                                                              uint8_t* __restrict__ codes, int64_t ldc,
                                                              uint8_t* __restrict__ scales, int64_t tiles_k, uint32_t runs,
                                                              int log_x) {
    begin_after_previous();
    const TensorFactor g((kFormat == DGA_NVFP4 && factor != nullptr) ? __ldg(factor) : 1.0f);
    // 2^log_x threads along a row, the block's others on the rows below
    const uint32_t run = (blockIdx.x << log_x) + (threadIdx.x & ((1u << log_x) - 1));
    const int64_t k = static_cast<int64_t>(run) * 32;
    // runs past the last value, up to the end of its scale tile: scales of 0
    if (run >= runs) return;
    const uint32_t rows_per_block = 256u >> log_x;
    const uintptr_t begin = reinterpret_cast<uintptr_t>(X), end = begin + ((rows - 1) * ldx + K) * sizeof(T);
    for (uint32_t r = blockIdx.y * rows_per_block + (threadIdx.x >> log_x); r < rows; r += gridDim.y * rows_per_block) {
        const T* src = X + static_cast<int64_t>(r) * ldx + k;
        uint32_t w[16];
        if (vec && k + 32 <= K) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + q);
                w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
            }
        } else if (reinterpret_cast<uintptr_t>(src) - begin >= 16 && reinterpret_cast<uintptr_t>(src) + 80 <= end) {
            // (begin, end: of X's bytes; a piece may hold neighbours of the row)
            load_words_shifted(src, w);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                if (k + 2 * q >= K) w[q] = 0;
                else if (k + 2 * q + 1 >= K) w[q] &= 0xffffu;
            }
        } else {
            const uint16_t* bits = reinterpret_cast<const uint16_t*>(src);
#pragma unroll
            for (int q = 0; q < 16; ++q)
                w[q] = (k + 2 * q < K ? static_cast<uint32_t>(bits[2 * q]) : 0u) |
                       (k + 2 * q + 1 < K ? static_cast<uint32_t>(bits[2 * q + 1]) << 16 : 0u);
        }
        constexpr int kPer = 32 / mx_block(kFormat);  // blocks of a thread
        uint4 out;
        uint32_t bytes;
        quantize_run16<kFormat, T>(w, g, out, bytes);  // past the last value: zero codes and scales
        if (k < K) *reinterpret_cast<uint4*>(codes + static_cast<int64_t>(r) * ldc + (k >> 1)) = out;
        uint8_t* dst = scales + mx_scale_offset(r, static_cast<int64_t>(run) * kPer, tiles_k);
        if constexpr (kPer == 1) *dst = static_cast<uint8_t>(bytes);
        else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(bytes);
    }
}

template <int kFormat>
__global__ void __launch_bounds__(256) mx_quant_rows32_kernel(const float* __restrict__ X, int64_t ldx,
                                                            int64_t rows, int64_t K, bool vec,
                                                            const float* __restrict__ factor,
                                                            uint8_t* __restrict__ codes,
                                                            int64_t ldc, uint8_t* __restrict__ scales,
                                                            int64_t tiles_k, int64_t chunks,
                                                            int64_t row_bytes) {
    begin_after_previous();
    constexpr int kLanes = mx_block(kFormat) / 8;  // lanes of a block
    const int lane = threadIdx.x & 31;
    const TensorFactor g((kFormat == DGA_NVFP4 && factor != nullptr) ? __ldg(factor) : 1.0f);
    const int64_t total = rows * chunks;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); u < total;
         u += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t r = u / chunks, k = (u - r * chunks) * 256 + lane * 8;
        float x[8];
        load8(X + r * ldx, k, K, vec, x);
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, mag_bits(x[q]));
#pragma unroll
        for (int d = 1; d < kLanes; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
        const BlockScale b = block_scale<kFormat>(m, g);
        over_unit8<kFormat>(x, b);
        if ((k >> 1) < row_bytes) *reinterpret_cast<uint32_t*>(codes + r * ldc + (k >> 1)) = codes8(x);
        // four blocks' scales to the first lane of the four; a block past the
        // row's end has scale 0 (its codes are 0 too)
        uint32_t w = k < K ? b.byte : 0u;
        w |= __shfl_down_sync(0xffffffffu, w, kLanes) << 8;
        w |= __shfl_down_sync(0xffffffffu, w, 2 * kLanes) << 16;
        const int64_t s = k / mx_block(kFormat);
        if (lane % (4 * kLanes) == 0 && (s >> 2) < tiles_k)
            *reinterpret_cast<uint32_t*>(scales + mx_scale_offset(r, s, tiles_k)) = w;
    }
}

// ---- along columns -----------------------------------------------------------
//
// The transpose of X (rows x cols) in 4 bits: cols rows of K = rows values.  A
// CTA takes 128 (k) x 128 (columns) of X, a thread 32 k of one column (fp32) or
// of two adjacent ones (16 bits), read straight from memory (a warp 128
// consecutive bytes) with all 32 loads under way at once.  Codes and scales go
// out through shared memory, so that each row of the result gets 64 consecutive
// bytes and scales are written as whole tiles.  8192 x 8192 MXFP4: bf16 31 us,
// fp32 52 us; with X's tile through shared memory 51 and 81 us.

// The end of both kernels: codes of 128 rows x 128 k, and their scale tiles.
template <int kFormat>
__device__ __forceinline__ void cols_out(const uint32_t (&out)[128][16 + 4], const uint8_t* tiles, int t, int threads, int64_t k0,
                                         int64_t c0, int64_t cols, uint8_t* __restrict__ codes, int64_t ldc,
                                         uint8_t* __restrict__ scales, int64_t tiles_k, int64_t row_bytes) {
    constexpr int kTiles = 32 / mx_block(kFormat);
    const int64_t first_tile = k0 / 128 * kTiles;
    if (t < kTiles * (kMxTileBytes / 16) && first_tile + t / (kMxTileBytes / 16) < tiles_k)
        reinterpret_cast<uint4*>(scales + mx_scale_offset(c0, first_tile * 4, tiles_k))[t] = reinterpret_cast<const uint4*>(tiles)[t];
    for (int idx = t; idx < 512; idx += threads) {
        const int orow = idx >> 2, ow = (idx & 3) * 4;  // 16 bytes of a result row
        const int64_t byte = (k0 >> 1) + ow * 4;
        if (c0 + orow < cols && byte < row_bytes)
            *reinterpret_cast<uint4*>(codes + (c0 + orow) * ldc + byte) = *reinterpret_cast<const uint4*>(&out[orow][ow]);
    }
}

template <int kFormat>
__global__ void __launch_bounds__(512) mx_quant_cols32_kernel(const float* __restrict__ X, int64_t ldx, int64_t K, int64_t cols,
                                                              const float* __restrict__ factor, uint8_t* __restrict__ codes,
                                                              int64_t ldc, uint8_t* __restrict__ scales, int64_t tiles_k,
                                                              int64_t blocks_k, int64_t row_bytes) {
    begin_after_previous();
    __shared__ __align__(16) uint32_t out[128][16 + 4];
    constexpr int kB = mx_block(kFormat), kPer = 32 / kB;
    __shared__ __align__(16) uint8_t tiles[kPer * kMxTileBytes];
    const int t = threadIdx.x, col = t & 127, quarter = t >> 7;
    const int64_t k0 = (blockIdx.x % blocks_k) * 128, c0 = (blockIdx.x / blocks_k) * 128;
    const TensorFactor g((kFormat == DGA_NVFP4 && factor != nullptr) ? __ldg(factor) : 1.0f);
    const int64_t k = k0 + quarter * 32;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(X + k * ldx + c0 + col);
    uint32_t raw[32];
    if (k + 32 <= K && c0 + col < cols) {
#pragma unroll
        for (int q = 0; q < 32; ++q) raw[q] = __ldg(src + q * ldx);
    } else {
#pragma unroll
        for (int q = 0; q < 32; ++q) raw[q] = k + q < K && c0 + col < cols ? __ldg(src + q * ldx) : 0u;
    }
    uint4 four;
    uint32_t bytes;
    quantize_run<kFormat>(DGA_F32, raw, g, four, bytes);
    // blocks past the last value have a scale of 0
#pragma unroll
    for (int p = 0; p < kPer; ++p)
        if (k + p * kB >= K) bytes &= ~(0xffu << (8 * p));
    *reinterpret_cast<uint4*>(&out[col][quarter * 4]) = four;
    uint8_t* dst = tiles + mx_scale_offset(col, quarter * kPer, kPer);
    if constexpr (kPer == 1) *dst = static_cast<uint8_t>(bytes);
    else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(bytes);
    __syncthreads();
    cols_out<kFormat>(out, tiles, t, 512, k0, c0, cols, codes, ldc, scales, tiles_k, row_bytes);
}

// (of 16-bit sources, where rows start on a word; their two maxima are taken
// together)
template <int kFormat, typename T>
__global__ void __launch_bounds__(256) mx_quant_cols16_kernel(const T* __restrict__ X, int64_t ldx,
                                                              int64_t K, int64_t cols, bool vec,
                                                              const float* __restrict__ factor,
                                                              uint8_t* __restrict__ codes,
                                                              int64_t ldc, uint8_t* __restrict__ scales,
                                                              int64_t tiles_k, int64_t blocks_k,
                                                              int64_t row_bytes) {
    begin_after_previous();
    __shared__ __align__(16) uint32_t out[128][16 + 4];
    // the scales of 128 rows and 128 k: one tile (MXFP4) or two, which lie together
    constexpr int kTiles = 32 / mx_block(kFormat);
    __shared__ __align__(16) uint8_t tiles[kTiles * kMxTileBytes];
    const int t = threadIdx.x;
    const int64_t k0 = (blockIdx.x % blocks_k) * 128, c0 = (blockIdx.x / blocks_k) * 128;
    const TensorFactor g((kFormat == DGA_NVFP4 && factor != nullptr) ? __ldg(factor) : 1.0f);
    const int pair = t & 63, quarter = t >> 6;
    constexpr int kB = mx_block(kFormat), kPer = 32 / kB;
    uint32_t all[32];
    {
        const int64_t k = k0 + quarter * 32, c = c0 + 2 * pair;
        const uint16_t* src = reinterpret_cast<const uint16_t*>(X + k * ldx + c);
        if (vec && k + 32 <= K && c + 2 <= cols) {
#pragma unroll
            for (int q = 0; q < 32; ++q) all[q] = __ldg(reinterpret_cast<const uint32_t*>(src + q * ldx));
        } else {
#pragma unroll
            for (int q = 0; q < 32; ++q)
                all[q] = (k + q < K && c < cols ? static_cast<uint32_t>(src[q * ldx]) : 0u) |
                         (k + q < K && c + 1 < cols ? static_cast<uint32_t>(src[q * ldx + 1]) << 16 : 0u);
        }
    }
    uint32_t four[2][4], word[2] = {0, 0};
#pragma unroll
    for (int p = 0; p < kPer; ++p) {
        const uint32_t* w = all + p * kB;
        uint32_t m2 = 0;
#pragma unroll
        for (int q = 0; q < kB; ++q) m2 = max_mag2(m2, w[q]);
        const int64_t k = k0 + quarter * 32 + p * kB;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const BlockScale b = block_scale<kFormat>(mag_bits(half_value<T>(m2, h)), g);
#pragma unroll
            for (int o = 0; o < kB / 8; ++o) {
                float y[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) y[q] = half_value<T>(w[o * 8 + q], h);
                over_unit8<kFormat>(y, b);
                four[h][p * (kB / 8) + o] = codes8(y);
            }
            word[h] |= (k < K ? static_cast<uint32_t>(b.byte) : 0u) << (8 * p);
        }
    }
    const int s = quarter * kPer;  // of the blocks in these 128 k
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int c = 2 * pair + h;
        *reinterpret_cast<uint4*>(&out[c][quarter * 4]) = make_uint4(four[h][0], four[h][1], four[h][2], four[h][3]);
        uint8_t* dst = tiles + mx_scale_offset(c, s, kTiles);
        if constexpr (kPer == 1) *dst = static_cast<uint8_t>(word[h]);
        else *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(word[h]);
    }
    __syncthreads();
    cols_out<kFormat>(out, tiles, t, 256, k0, c0, cols, codes, ldc, scales, tiles_k, row_bytes);
}

// ---- back to values ------------------------------------------------------------

template <typename T>
__device__ __forceinline__ T mx_out(float v);
template <> __device__ __forceinline__ float mx_out<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 mx_out<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half mx_out<__half>(float v) { return __float2half_rn(v); }

__device__ __forceinline__ float scale_value(int format, uint8_t byte) {
    if (format == DGA_MXFP4)  // 2^(byte - 127): byte 0 is the subnormal 2^-127, 255 NaN
        return byte == 0 ? __uint_as_float(0x00400000u)
                         : (byte == 255 ? __uint_as_float(0x7fffffffu) : __uint_as_float(static_cast<uint32_t>(byte) << 23));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h2 & 0xffff)));
}

// A lane makes 16 bytes of a row, code times (scale times factor) in fp32
// rounded to the output type, for several rows of the same columns.  Bound
// by memory (0.53 bytes in, 2 or 4 out a value), so four rows' loads go out
// before the first is used: 8192 x 8192 in 31 us to bf16 (5.5 TB/s), 51 us to
// fp32 (5.9 TB/s; 54 us with a 64-bit division and one row at a time, 65 us with
// eight values, two separate stores, to a lane).
// kShifted: rows do not start on 16 bytes; the pieces, of eight values, begin
// at the first aligned address at or before a row's start, and their codes lie
// across two words and maybe two blocks (4093 x 4099:
// bf16 17 us against 51 us with element stores, fp32 21 us against 25 us).
constexpr int kDequantRows = 4;
template <int kFormat, typename T, bool kShifted>
__global__ void __launch_bounds__(256) mx_dequant_kernel(uint32_t rows, int32_t K, const uint8_t* __restrict__ codes, int64_t ldc,
                                                         const uint8_t* __restrict__ scales, int64_t tiles_k,
                                                         const float* __restrict__ factor, T* __restrict__ Y, int64_t ldy,
                                                         int log_x) {
    constexpr int kAlign = 16 / sizeof(T), kPer = kShifted ? 8 : kAlign, kBlock = mx_block(kFormat);
    begin_after_previous();
    const float g = (kFormat == DGA_NVFP4 && factor != nullptr) ? __ldg(factor) : 1.0f;
    // 2^log_x threads along a row, the block's others on the rows below
    const int32_t piece = static_cast<int32_t>((blockIdx.x << log_x) + (threadIdx.x & ((1u << log_x) - 1))) * kPer;
    const uint32_t step = gridDim.y * (256u >> log_x);
    for (uint32_t r0 = blockIdx.y * (256u >> log_x) + (threadIdx.x >> log_x); r0 < rows; r0 += step * kDequantRows) {
        int32_t k[kDequantRows];  // the piece's first column, below 0 or past K where it is not a whole one
        uint32_t c[kDequantRows];
        uint8_t scale[kDequantRows], scale2[kDequantRows];
#pragma unroll
        for (int i = 0; i < kDequantRows; ++i) {
            const uint32_t r = r0 + i * step;
            k[i] = piece;
            if constexpr (kShifted)
                k[i] -= static_cast<int32_t>(reinterpret_cast<uintptr_t>(Y + static_cast<int64_t>(r) * ldy) / sizeof(T) & (kAlign - 1));
            if (r >= rows || k[i] >= K) continue;
            const uint32_t first = max(k[i], 0), last = min(k[i] + kPer, K) - 1;
            const uint8_t* src = codes + static_cast<int64_t>(r) * ldc;
            if constexpr (kShifted) {
                // nibbles k .. k + kPer - 1, the first at bit 0 (those below 0 or past K are not used)
                const uint32_t w0 = first >> 3, w1 = last >> 3;
                const uint32_t* words = reinterpret_cast<const uint32_t*>(src);
                const uint32_t lo = __ldg(words + w0), hi = w1 > w0 ? __ldg(words + w1) : 0;
                c[i] = k[i] < 0 ? lo << (static_cast<uint32_t>(-k[i]) * 4) : __funnelshift_r(lo, hi, (static_cast<uint32_t>(k[i]) & 7) * 4);
            } else if constexpr (kPer == 8) {
                c[i] = __ldg(reinterpret_cast<const uint32_t*>(src + (first >> 1)));
            } else {
                c[i] = __ldg(reinterpret_cast<const uint16_t*>(src + (first >> 1)));
            }
            scale[i] = __ldg(scales + mx_scale_offset(r, first / kBlock, tiles_k));
            if constexpr (kShifted) scale2[i] = __ldg(scales + mx_scale_offset(r, last / kBlock, tiles_k));
        }
#pragma unroll
        for (int i = 0; i < kDequantRows; ++i) {
            const uint32_t r = r0 + i * step;
            if (r >= rows || k[i] >= K) continue;
            float v[8];
            values8(c[i], v);
            const float s = scale_value(kFormat, scale[i]) * g, s2 = kShifted ? scale_value(kFormat, scale2[i]) * g : s;
            // values from this one on belong to the second block
            const int turn = (k[i] + kPer - 1) / kBlock * kBlock - k[i];
            T y[kPer];
#pragma unroll
            for (int q = 0; q < kPer; ++q) y[q] = mx_out<T>(v[q] * (kShifted && turn > 0 && q >= turn && k[i] >= 0 ? s2 : s));
            T* dst = Y + static_cast<int64_t>(r) * ldy + k[i];
            if (k[i] >= 0 && k[i] + kPer <= K) {
                uint4 x[kPer / kAlign];
                memcpy(x, y, sizeof x);
#pragma unroll
                for (int q = 0; q < kPer / kAlign; ++q) reinterpret_cast<uint4*>(dst)[q] = x[q];
            } else {
#pragma unroll
                for (int q = 0; q < kPer; ++q)
                    if (k[i] + q >= 0 && k[i] + q < K) dst[q] = y[q];
            }
        }
    }
}

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kern)(P...), dim3 grid, unsigned threads, cudaStream_t stream, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

template <int kFormat, typename T>
cudaError_t quantize_as(const MxQuantArgs& a, const DeviceInfo& dev) {
    const T* X = static_cast<const T*>(a.X);
    constexpr int64_t kVec = 16 / sizeof(T);
    const bool vec = aligned(a.X, 16) && a.ldx % kVec == 0;
    const int64_t K = a.transpose ? a.rows : a.cols;
    const int64_t tiles_k = mx_tiles_k(kFormat, K), row_bytes = mx_row_bytes(K);
    if (!a.transpose) {
        if constexpr (sizeof(T) == 2) {
            // runs of 32 values, to the end of the last scale tile
            const int64_t runs = tiles_k * 4 * mx_block(kFormat) / 32;
            int log_x = 0;
            while (log_x < 8 && (int64_t{1} << log_x) < runs) ++log_x;
            const int64_t rows_per_block = 256 >> log_x;
            const dim3 grid(static_cast<unsigned>((runs + (1 << log_x) - 1) >> log_x),
                            static_cast<unsigned>(std::min<int64_t>((a.rows + rows_per_block - 1) / rows_per_block, 65535)));
            return launch_behind(mx_quant_rows16_kernel<kFormat, T>, grid, 256, a.stream, X, a.ldx, static_cast<uint32_t>(a.rows), K,
                                 vec, a.factor, a.codes, a.ld_codes, a.scales, tiles_k, static_cast<uint32_t>(runs), log_x);
        } else {
            const int64_t chunks = (K + 255) / 256, units = a.rows * chunks;
            const int64_t blocks = std::min<int64_t>((units + 7) / 8, static_cast<int64_t>(dev.sm_count) * 64);
            return launch_behind(mx_quant_rows32_kernel<kFormat>, dim3(static_cast<unsigned>(blocks)), 256, a.stream, X, a.ldx,
                                 a.rows, K, vec, a.factor, a.codes, a.ld_codes, a.scales, tiles_k, chunks, row_bytes);
        }
    } else {
        const int64_t blocks_k = (K + 127) / 128, blocks = blocks_k * ((a.cols + 127) / 128);
        if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
        const dim3 grid(static_cast<unsigned>(blocks));
        if constexpr (sizeof(T) == 2) {
            // two values of a row at once
            const bool pairs = aligned(a.X, 4) && a.ldx % 2 == 0;
            return launch_behind(mx_quant_cols16_kernel<kFormat, T>, grid, 256, a.stream, X, a.ldx, K, a.cols, pairs, a.factor,
                                 a.codes, a.ld_codes, a.scales, tiles_k, blocks_k, row_bytes);
        } else {
            return launch_behind(mx_quant_cols32_kernel<kFormat>, grid, 512, a.stream, X, a.ldx, K, a.cols, a.factor, a.codes,
                                 a.ld_codes, a.scales, tiles_k, blocks_k, row_bytes);
        }
    }
}

template <int kFormat, typename T>
cudaError_t dequantize_as(const MxMatrix& q, int64_t rows, int64_t K, void* Y, int64_t ldy,
                          const DeviceInfo& dev, cudaStream_t stream) {
    constexpr int64_t kVec = 16 / sizeof(T);
    const bool vec = aligned(Y, 16) && ldy % kVec == 0;
    const int64_t groups = vec ? (K + kVec - 1) / kVec : (K + 7) / 8 + 1;
    int log_x = 0;
    while (log_x < 8 && (int64_t{1} << log_x) < groups) ++log_x;
    const int64_t per_block = 256 >> log_x, cols = (groups + (int64_t{1} << log_x) - 1) >> log_x;
    const int64_t all = (rows + per_block - 1) / per_block;  // blocks that a column of them needs, a row to a thread
    // several rows to a thread once the machine is full
    const int64_t down = cols * all >= static_cast<int64_t>(dev.sm_count) * 8 * kDequantRows ? (all + kDequantRows - 1) / kDequantRows : all;
    const dim3 grid(static_cast<unsigned>(cols), static_cast<unsigned>(std::min<int64_t>(down, 65535)));
    const auto kernel = vec ? mx_dequant_kernel<kFormat, T, false> : mx_dequant_kernel<kFormat, T, true>;
    return launch_behind(kernel, grid, 256, stream, static_cast<uint32_t>(rows), static_cast<int32_t>(K), static_cast<const uint8_t*>(q.codes), q.ld,
                                     static_cast<const uint8_t*>(q.scales), mx_tiles_k(kFormat, K), q.factor, static_cast<T*>(Y),
                                     ldy, log_x);
}

}  // namespace

cudaError_t mx_quantize_launch(const MxQuantArgs& a, const DeviceInfo& dev) {
    const bool mx = a.format == DGA_MXFP4;
    switch (a.in_dtype) {
    case DGA_F32: return mx ? quantize_as<DGA_MXFP4, float>(a, dev) : quantize_as<DGA_NVFP4, float>(a, dev);
    case DGA_BF16: return mx ? quantize_as<DGA_MXFP4, __nv_bfloat16>(a, dev) : quantize_as<DGA_NVFP4, __nv_bfloat16>(a, dev);
    default: return mx ? quantize_as<DGA_MXFP4, __half>(a, dev) : quantize_as<DGA_NVFP4, __half>(a, dev);
    }
}

cudaError_t mx_dequantize_launch(int format, int out_dtype, const MxMatrix& q, int64_t rows, int64_t K,
                                 void* Y, int64_t ldy, const DeviceInfo& dev, cudaStream_t stream) {
    const bool mx = format == DGA_MXFP4;
    switch (out_dtype) {
    case DGA_F32: return mx ? dequantize_as<DGA_MXFP4, float>(q, rows, K, Y, ldy, dev, stream) : dequantize_as<DGA_NVFP4, float>(q, rows, K, Y, ldy, dev, stream);
    case DGA_BF16: return mx ? dequantize_as<DGA_MXFP4, __nv_bfloat16>(q, rows, K, Y, ldy, dev, stream) : dequantize_as<DGA_NVFP4, __nv_bfloat16>(q, rows, K, Y, ldy, dev, stream);
    default: return mx ? dequantize_as<DGA_MXFP4, __half>(q, rows, K, Y, ldy, dev, stream) : dequantize_as<DGA_NVFP4, __half>(q, rows, K, Y, ldy, dev, stream);
    }
}

}  // namespace dga
