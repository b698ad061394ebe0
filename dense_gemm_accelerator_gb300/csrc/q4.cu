// q4.cu -- 4-bit weights with group scales: to that form and back to values.
//
//   w = (q - z) * s,  q and z in 0..15, a scale s (bf16 or fp16) and a zero
//   point z (a byte, or 8 throughout) per row and group of 32, 64 or 128 columns
//
// 8192 x 8192, groups of 128, bf16: back to values in 42.5 us, 4 TB/s.  To codes it takes
// 149 us (groups of 64: 217, of 32: 363) where the bytes take 25: the instructions of a
// warp to a group, a lane one to four values, fill 83 % of the issue slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "gated_act.cuh"

namespace dga {
namespace {

// A warp to a group, a lane kGroup / 32 consecutive values of it.
template <typename T, typename TS, int kGroup>
__global__ void __launch_bounds__(256)
    q4_quantize_kernel(int64_t rows, int64_t cols, const T* __restrict__ W, int64_t ldw, uint8_t* __restrict__ codes,
                       int64_t ld, TS* __restrict__ scales, int64_t lds, uint8_t* __restrict__ zeros, int64_t ldz) {
    constexpr int kPer = kGroup / 32;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (cols + kGroup - 1) / kGroup, padded = (cols + 31) / 32 * 32;
    const int64_t total = rows * groups, step = static_cast<int64_t>(gridDim.x) * 8;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total; i += step) {
        const int64_t row = i / groups, group = i - row * groups;
        const int64_t k0 = group * kGroup + lane * kPer;
        float w[kPer], lo = 0.0f, hi = 0.0f;
        bool finite = true;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            w[j] = k0 + j < cols ? static_cast<float>(W[row * ldw + k0 + j]) : 0.0f;
            lo = fminf(lo, w[j]);
            hi = fmaxf(hi, w[j]);
            finite = finite && fabsf(w[j]) <= 3.4028234663852886e38f;  // false for a NaN
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
        }
        finite = __all_sync(0xffffffffu, finite);
        TS held;
        OutT<TS>::store(&held, zeros ? __fdiv_rn(__fsub_rn(hi, lo), 15.0f) : __fdiv_rn(fmaxf(hi, -lo), 7.0f));
        const float s = OutT<TS>::load(&held);
        finite = finite && fabsf(s) <= 3.4028234663852886e38f;
        float z = 8.0f;
        if (zeros) z = finite && s > 0.0f ? fminf(15.0f, rintf(__fdiv_rn(-lo, s))) : 0.0f;
        uint32_t code = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            float q = z;
            if (finite && s > 0.0f) q = fmaxf(0.0f, fminf(15.0f, rintf(__fadd_rn(__fdiv_rn(w[j], s), z))));
            if (k0 + j < cols) code |= static_cast<uint32_t>(q) << (4 * j);
        }
        uint8_t* at = codes + row * ld + k0 / 2;
        if constexpr (kPer == 1) code |= __shfl_down_sync(0xffffffffu, code, 1) << 4;
        if (k0 < padded) {
            if constexpr (kPer == 4) *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(code);
            else if (kPer == 2 || (lane & 1) == 0) *at = static_cast<uint8_t>(code);
        }
        if (lane == 0) {
            OutT<TS>::store(scales + row * lds + group, finite ? s : __int_as_float(0x7fffffff));
            if (zeros) zeros[row * ldz + group] = static_cast<uint8_t>(z);
        }
    }
}

// A thread a word of codes, eight values; the grid's y walks the rows, four at a
// time with their loads together (a row's division out of one index took longer
// than the copy).  The gated layer's kernel behind it is a programmatic dependent;
// the GEMM is one only where it repacks X first, else an ordinary launch.
template <typename TS, typename T, bool kVec>
__global__ void __launch_bounds__(256)
    q4_dequantize_kernel(int64_t rows, int64_t cols, Q4Matrix q, int shift, T* __restrict__ Y, int64_t ldy) {
    constexpr int kRows = 4;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t k = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
    if (k >= cols) return;
    const int64_t group = k >> shift;
    const TS* scales = static_cast<const TS*>(q.scales) + group;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRows; row0 < rows; row0 += static_cast<int64_t>(gridDim.y) * kRows) {
        uint32_t c[kRows];
        float s[kRows], z[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t row = min(row0 + r, rows - 1);
            c[r] = __ldg(reinterpret_cast<const uint32_t*>(q.codes + row * q.ld + k / 2));
            s[r] = OutT<TS>::load(scales + row * q.ld_scales);
            z[r] = q.zeros ? static_cast<float>(__ldg(q.zeros + row * q.ld_zeros + group) & 15) : 8.0f;
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (row0 + r >= rows) break;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (static_cast<float>((c[r] >> (4 * j)) & 15u) - z[r]) * s[r];
            T* out = Y + (row0 + r) * ldy + k;
            if (kVec && k + 8 <= cols) {
                if constexpr (sizeof(T) == 2) {
                    Pack<T, 8>::store(out, v);
                } else {
                    const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
                    Pack<T, 4>::store(out, a);
                    Pack<T, 4>::store(out + 4, b);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k + j < cols) OutT<T>::store(out + j, v[j]);
            }
        }
    }
}

int group_shift(int group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

template <typename Fn>
cudaError_t for_float(int dtype, Fn&& f) {
    switch (dtype) {
    case DGA_F32: return f(float{});
    case DGA_BF16: return f(__nv_bfloat16{});
    case DGA_F16: return f(__half{});
    default: return cudaErrorInvalidValue;
    }
}
template <typename Fn>
cudaError_t for_half(int dtype, Fn&& f) {
    return dtype == DGA_BF16 ? f(__nv_bfloat16{}) : f(__half{});
}

unsigned blocks_for(int64_t work, int64_t per, const DeviceInfo& dev) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((work + per - 1) / per, int64_t{64} * dev.sm_count)));
}

}  // namespace

cudaError_t q4_quantize_launch(int in_dtype, int scale_dtype, int64_t rows, int64_t cols, const void* W, int64_t ldw,
                               const Q4Matrix& q, const DeviceInfo& dev, cudaStream_t stream) {
    const unsigned grid = blocks_for(rows * ((cols + q.group - 1) / q.group), 8, dev);
    return for_float(in_dtype, [&](auto t) {
        return for_half(scale_dtype, [&](auto ts) {
            using T = decltype(t);
            using TS = decltype(ts);
            auto kern = q.group == 32 ? q4_quantize_kernel<T, TS, 32>
                        : q.group == 64 ? q4_quantize_kernel<T, TS, 64> : q4_quantize_kernel<T, TS, 128>;
            kern<<<grid, 256, 0, stream>>>(rows, cols, static_cast<const T*>(W), ldw, const_cast<uint8_t*>(q.codes), q.ld,
                                           static_cast<TS*>(const_cast<void*>(q.scales)), q.ld_scales,
                                           const_cast<uint8_t*>(q.zeros), q.ld_zeros);
            return cudaGetLastError();
        });
    });
}

cudaError_t q4_dequantize_launch(int scale_dtype, int out_dtype, int64_t rows, int64_t cols, const Q4Matrix& q, void* Y,
                                 int64_t ldy, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((cols + 2047) / 2048), static_cast<unsigned>(std::min<int64_t>((rows + 3) / 4, 65535)));
    const bool vec = aligned(Y, 16) && ldy % 8 == 0;
    return for_half(scale_dtype, [&](auto ts) {
        return for_float(out_dtype, [&](auto t) {
            using T = decltype(t);
            using TS = decltype(ts);
            auto kern = vec ? q4_dequantize_kernel<TS, T, true> : q4_dequantize_kernel<TS, T, false>;
            kern<<<grid, 256, 0, stream>>>(rows, cols, q, group_shift(q.group), static_cast<T*>(Y), ldy);
            return cudaGetLastError();
        });
    });
}

}  // namespace dga
