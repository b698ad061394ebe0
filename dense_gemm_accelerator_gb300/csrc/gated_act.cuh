// gated_act.cuh -- the gated layer's activations and their slopes, and the
// 16-bit vectors that its kernels load and store.
//
//   silu       g s(g)          s(g) = 1 / (1 + e^-g)
//   gelu       g Phi(g)        Phi(g) = (1 + erf(g / sqrt 2)) / 2
//   gelu_tanh  g s(v)          v = 2 sqrt(2/pi) (g + 0.044715 g^3), since
//                              (1 + tanh(v / 2)) / 2 = s(v)
//   relu       max(g, 0)
//   sigmoid    s(g)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "dga.h"

namespace dga {

// s(x) and its complement s(-x) = 1 - s(x).  With e = e^-|x| and r = 1 / (1 + e) the
// larger of the two is r and the smaller e r, so neither is a difference: 1 - s, which is
// what sigmoid's slope s (1 - s) would take, has lost 9e-3 of itself in fp32 at x = 12 and
// is 0 from 17 on.  Nor is there an infinity for large -x.
// kFast: the hardware's exponential and division, for results that are rounded to 16 bits
// (2^-9, 2^-12) next.  The larger is 2^-21 off, the smaller 2^-20 + 1.2 |x| 2^-23 (the
// exponential's error grows with its argument: 2^-16 at |x| = 88).
template <bool kFast>
__device__ __forceinline__ float2 logistic_pair(float x) {
    const float e = kFast ? __expf(-fabsf(x)) : expf(-fabsf(x));
    const float r = kFast ? __fdividef(1.0f, 1.0f + e) : 1.0f / (1.0f + e);
    return x < 0.0f ? make_float2(e * r, r) : make_float2(r, e * r);
}
template <bool kFast>
__device__ __forceinline__ float logistic(float x) { return logistic_pair<kFast>(x).x; }

// Phi(g).  kFast: erfc(x) = t 2^(-x^2 log2 e + p(t)), t = 1 / (1 + x / 2), x = |g| / sqrt 2,
// p the polynomial of degree 7 that a Chebyshev fit of log2(erfcx(x) / t) over t gives;
// 7e-7 off relative to the value near 0, 2e-5 at |g| = 13 (fp32's x^2), where the library
// function (the other case) took three times the tensor cores' time of K = 512.
template <bool kFast>
__device__ __forceinline__ float normal_cdf(float g) {
    if constexpr (!kFast) return normcdff(g);
    const float x = fabsf(g) * 0.70710678f, t = __fdividef(1.0f, fmaf(0.5f, x, 1.0f));
    float q = -0.2702641784782f;
    q = fmaf(q, t, 1.0810290575f);
    q = fmaf(q, t, -1.4374856949f);
    q = fmaf(q, t, 0.4973544180f);
    q = fmaf(q, t, -0.0525670536f);
    q = fmaf(q, t, 0.5666871667f);
    q = fmaf(q, t, 1.4409651756f);
    q = fmaf(q, t, -1.8257199526f);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(-1.44269504f * x, x, q)));
    e *= 0.5f * t;
    return g < 0.0f ? e : 1.0f - e;
}

constexpr float kGeluA = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluB = 0.071354816272600f;    // 0.044715 * kGeluA
constexpr float kGeluC = 0.21406444881780f;     // 3 * kGeluB
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int kAct, bool kFast>
__device__ __forceinline__ float act_value(float g) {
    if constexpr (kAct == DGA_SILU) return g * logistic<kFast>(g);
    else if constexpr (kAct == DGA_GELU) return g * normal_cdf<kFast>(g);
    else if constexpr (kAct == DGA_GELU_TANH) return g * logistic<kFast>(g * fmaf(kGeluB * g, g, kGeluA));
    else if constexpr (kAct == DGA_RELU) return g < 0.0f ? 0.0f : g;  // a NaN stays one
    else return logistic<kFast>(g);
}

// The value and the slope.
template <int kAct, bool kFast>
__device__ __forceinline__ void act_both(float g, float& value, float& slope) {
    if constexpr (kAct == DGA_SILU) {
        const float2 s = logistic_pair<kFast>(g);
        value = g * s.x;
        slope = fmaf(value, s.y, s.x);
    } else if constexpr (kAct == DGA_GELU) {
        const float c = normal_cdf<kFast>(g);
        const float e = kInvSqrt2Pi * (kFast ? __expf(-0.5f * g * g) : expf(-0.5f * g * g));
        value = g * c;
        slope = fmaf(g, e, c);
    } else if constexpr (kAct == DGA_GELU_TANH) {
        const float2 s = logistic_pair<kFast>(g * fmaf(kGeluB * g, g, kGeluA));
        const float t = s.x * s.y;
        value = g * s.x;
        // far out t is 0 and v' past fp32's range
        slope = t > 0.0f ? fmaf(g * t, fmaf(kGeluC * g, g, kGeluA), s.x) : s.x;
    } else if constexpr (kAct == DGA_RELU) {
        value = g < 0.0f ? 0.0f : g;
        slope = g > 0.0f ? 1.0f : (g == g ? 0.0f : g);
    } else {
        const float2 s = logistic_pair<kFast>(g);
        value = s.x;
        slope = s.x * s.y;
    }
}

// kVec values of T, loaded and stored as one access.
template <typename T, int kVec>
struct Pack {
    static constexpr int kBytes = kVec * static_cast<int>(sizeof(T));
    __device__ __forceinline__ static void load(const T* p, float (&v)[kVec]) {
        T t[kVec];
        if constexpr (kBytes == 16) {
            const uint4 w = *reinterpret_cast<const uint4*>(p);
            memcpy(t, &w, 16);
        } else if constexpr (kBytes == 8) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            memcpy(t, &w, 8);
        } else {
            static_assert(kVec == 1, "16 or 8 bytes, or one value");
            t[0] = *p;
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = static_cast<float>(t[i]);
    }
    __device__ __forceinline__ static void store(T* p, const float (&v)[kVec]) {
        T t[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
            if constexpr (sizeof(T) == 4) t[i] = v[i];
            else if constexpr (std::is_same<T, __half>::value) t[i] = __float2half_rn(v[i]);
            else t[i] = __float2bfloat16_rn(v[i]);
        }
        if constexpr (kBytes == 16) {
            uint4 w;
            memcpy(&w, t, 16);
            *reinterpret_cast<uint4*>(p) = w;
        } else if constexpr (kBytes == 8) {
            uint2 w;
            memcpy(&w, t, 8);
            *reinterpret_cast<uint2*>(p) = w;
        } else {
            *p = t[0];
        }
    }
};

}  // namespace dga
