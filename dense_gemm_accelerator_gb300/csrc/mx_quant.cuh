// mx_quant.cuh -- the roundings of the 4-bit formats (see mx_quant.cu), for the
// kernels that quantise: block scales, values over their unit, codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "mx_common.cuh"

namespace dga {

// Magnitude bits of x: ordered like |x|, with infinity and NaN on top.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// a / b, correctly rounded, from inv = 1 / b correctly rounded: the product,
// its residual and one correction (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  For b and a / b
// far enough from the ends of fp32's range that the residual is exact.
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    const float q = a * inv;
    return fmaf(fmaf(-q, b, a), inv, q);
}
__device__ __forceinline__ bool mid_range(float x) { return x >= 0x1p-90f && x <= 0x1p90f; }

// The plain division for the rest, out of line: it is hardly ever taken.
static __device__ __noinline__ float plain_quotient(float a, float b) { return __fdiv_rn(a, b); }

// What NVFP4's scales are found with: the tensor's factor g, and 6 g.
struct TensorFactor {
    float g, six, inv_six;
    bool plain;  // 6 g where quotient() does not hold
    __device__ __forceinline__ explicit TensorFactor(float factor) : g(factor) {
        six = __fmul_rn(6.0f, g);
        inv_six = __frcp_rn(six);
        plain = !mid_range(six);
    }
};

// One block's scale byte and what its values are divided by: MXFP4
// multiplies by `inv`, the exact 2^-e; NVFP4 divides by `unit`.
struct BlockScale {
    uint8_t byte;
    bool plain;  // quotient() does not hold for the unit, or the largest value over it
    float unit, inv;
};

template <int kFormat>
__device__ __forceinline__ BlockScale block_scale(uint32_t amax_bits, const TensorFactor& f) {
    BlockScale b;
    const bool finite = amax_bits < 0x7f800000u;
    if constexpr (kFormat == DGA_MXFP4) {
        // biased exponent of the scale: floor(log2 m) + 127 - 2, at least 0
        // (a subnormal m has exponent field 0); at most 252
        const uint32_t e = amax_bits >> 23;
        const uint32_t s = e > 2 ? e - 2 : 0;
        b.byte = finite ? static_cast<uint8_t>(s) : uint8_t(0xff);
        b.inv = finite ? __uint_as_float((254u - s) << 23) : 0.0f;
        b.unit = 0.0f;  // not used
        b.plain = false;
    } else {
        const float m = __uint_as_float(amax_bits);
        // Values that may pass fp32's range over the unit, of which quotient()
        // would make NaN: m / unit is above 12 only where the scale is held to
        // 448, and 6 / 448 of m / (6 g) there.
        const bool far = !(m * f.inv_six <= 0x1p90f);
        // (a zero block's scale is 0 whatever the factor, which of a zero tensor is 0 too)
        float r = m == 0.0f ? 0.0f : quotient(m, f.six, f.inv_six);
        if (m != 0.0f && (f.plain | far | (m < 0x1p-90f))) r = plain_quotient(m, f.six);
        uint16_t two;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two) : "f"(0.0f), "f"(r));
        b.byte = finite ? static_cast<uint8_t>(two & 0xff) : uint8_t(0x7f);
        uint32_t h2;  // the scale back as fp16 (exact)
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
        const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(h2 & 0xffff)));
        b.unit = finite ? __fmul_rn(s, f.g) : 0.0f;
        b.inv = b.unit > 0.0f ? __frcp_rn(b.unit) : 0.0f;
        b.plain = (b.unit != 0.0f) & (far | !mid_range(b.unit));  // 0: inv is 0 too, and so is the quotient
    }
    return b;
}

// Eight values over the block's unit, in place; a zero unit gives zeros of the
// values' signs.
template <int kFormat>
__device__ __forceinline__ void over_unit8(float (&x)[8], const BlockScale& b) {
    if constexpr (kFormat == DGA_MXFP4) {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] *= b.inv;
    } else if (!b.plain) {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = copysignf(quotient(x[q], b.unit, b.inv), x[q]);  // the sign of a zero too
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = plain_quotient(x[q], b.unit);
    }
}

// Eight values to eight codes, value i in bits 4i..4i+3.
__device__ __forceinline__ uint32_t codes8(const float (&t)[8]) {
    uint32_t out;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(out)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return out;
}

// Larger of the magnitudes (bits, ordered like the values) in each half.
__device__ __forceinline__ uint32_t max_mag2(uint32_t a, uint32_t b) {
    return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ float half_value(uint32_t word, int h);
template <>
__device__ __forceinline__ float half_value<__nv_bfloat16>(uint32_t word, int h) {
    return __uint_as_float(h ? word & 0xffff0000u : word << 16);
}
template <>
__device__ __forceinline__ float half_value<__half>(uint32_t word, int h) {
    return __half2float(__ushort_as_half(static_cast<uint16_t>(h ? word >> 16 : word)));
}

// 32 consecutive values of a row as raw bits, zero past its end (`left` values
// from `src` on): 16 words of two 16-bit values, or 32 of one fp32.
__device__ __forceinline__ void load_run(int type, const void* src, int64_t left, bool vec, uint32_t (&raw)[32]) {
    const int words = type == DGA_F32 ? 32 : 16;
    if (vec && left >= 32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (q * 4 < words) {
                const uint4 v = __ldg(static_cast<const uint4*>(src) + q);
                raw[4 * q] = v.x, raw[4 * q + 1] = v.y, raw[4 * q + 2] = v.z, raw[4 * q + 3] = v.w;
            }
        }
    } else if (type == DGA_F32) {
#pragma unroll
        for (int q = 0; q < 32; ++q) raw[q] = q < left ? static_cast<const uint32_t*>(src)[q] : 0u;
    } else {
        const uint16_t* bits = static_cast<const uint16_t*>(src);
#pragma unroll
        for (int q = 0; q < 16; ++q)
            raw[q] = (2 * q < left ? static_cast<uint32_t>(bits[2 * q]) : 0u) |
                     (2 * q + 1 < left ? static_cast<uint32_t>(bits[2 * q + 1]) << 16 : 0u);
    }
}

// Their 16 bytes of codes, and scale bytes (one block or two).
template <int kFormat, typename T>
__device__ __forceinline__ void quantize_run16(const uint32_t* w, const TensorFactor& g, uint4& codes, uint32_t& bytes) {
    constexpr int kB = mx_block(kFormat);
    uint32_t out[4];
    bytes = 0;
#pragma unroll
    for (int p = 0; p < 32 / kB; ++p) {
        uint32_t m2 = 0;
#pragma unroll
        for (int q = 0; q < kB / 2; ++q) m2 = max_mag2(m2, w[p * (kB / 2) + q]);
        // the larger half as fp32 bits (infinity and NaN stay what they are)
        const uint32_t m16 = max(m2 & 0xffffu, m2 >> 16);
        const BlockScale b = block_scale<kFormat>(mag_bits(half_value<T>(m16, 0)), g);
#pragma unroll
        for (int o = 0; o < kB / 8; ++o) {
            float t[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = half_value<T>(w[p * (kB / 2) + o * 4 + q / 2], q & 1);
            over_unit8<kFormat>(t, b);
            out[p * (kB / 8) + o] = codes8(t);
        }
        bytes |= static_cast<uint32_t>(b.byte) << (8 * p);
    }
    codes = make_uint4(out[0], out[1], out[2], out[3]);
}
template <int kFormat>
__device__ __forceinline__ void quantize_run(int type, const uint32_t (&raw)[32], const TensorFactor& g, uint4& codes,
                                             uint32_t& bytes) {
    if (type == DGA_BF16) return quantize_run16<kFormat, __nv_bfloat16>(raw, g, codes, bytes);
    if (type == DGA_F16) return quantize_run16<kFormat, __half>(raw, g, codes, bytes);
    constexpr int kB = mx_block(kFormat);
    uint32_t out[4];
    bytes = 0;
#pragma unroll
    for (int p = 0; p < 32 / kB; ++p) {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < kB; ++q) m = max(m, raw[p * kB + q] & 0x7fffffffu);
        const BlockScale b = block_scale<kFormat>(m, g);
#pragma unroll
        for (int o = 0; o < kB / 8; ++o) {
            float t[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) t[q] = __uint_as_float(raw[p * kB + o * 8 + q]);
            over_unit8<kFormat>(t, b);
            out[p * (kB / 8) + o] = codes8(t);
        }
        bytes |= static_cast<uint32_t>(b.byte) << (8 * p);
    }
    codes = make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace dga
