// mx_gemm.cu -- products of 4-bit microscaled matrices on the tensor cores.
//
//   C <- alpha * fA * fB * sum_k a(i,k) b(j,k) + beta * C + bias(j)
//
// a(i,k) and b(j,k) are E2M1 codes times their block scales, fA and fB the
// tensors' fp32 factors.  tcgen05.mma's block-scaled kinds multiply the codes
// and the scales inside the MMA and accumulate in fp32: the products of codes
// and scales are exact, so fp32 accumulation is the only rounding before the
// epilogue's.
//
// Two kernels, both fed by TMA (codes as 128-byte swizzle rows of 256 values;
// scale tiles of 512 bytes, moved on to tensor memory before the MMAs that use
// them):
//
//   pair    a cluster of two CTAs per 256 x 256 tile of C, persistent; for
//           many rows, where the tensor cores' rate is the bound
//   skinny  one CTA per 128 rows of B and all (up to 256) rows of A, with the
//           operands' roles swapped: B's rows fill the MMA's M = 128, A's rows
//           its N, so that a few rows of A waste nothing; the K axis is shared
//           by a cluster and its parts joined through distributed shared
//           memory in a fixed order.  For few rows the bytes of B are the
//           bound.
//
// Measured: 8192^3 to bf16 172 us MXFP4 (6.4 PFLOP/s), 193 us NVFP4, where the
// operands' way into shared memory alone takes 138 us (46 to 60 bytes a clock
// and SM).  8192 x 8192 weights: 100 rows 18.6 us, 256 rows 24.8 us (MXFP4);
// 13 rows of values 12.5 us MXFP4, 16.6 us NVFP4, of which the weight's 36 MB
// take 5.3 us at the copy rate.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "mx_common.cuh"
#include "mx_quant.cuh"
#include "ptx.cuh"

namespace dga {

__device__ int g_mx_status;  // non-zero: a bounded wait expired (role code)

namespace {

constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s
constexpr int kRowBytes = 128;                    // one stage of a row: 256 codes
constexpr int kStageK = 256;
enum : int { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3, kRoleScales = 4 };

// Scale tiles (4 blocks) of one stage's 256 values.
__host__ __device__ constexpr int scale_tiles(int format) { return kStageK / (4 * mx_block(format)); }

struct MxParams {
    int64_t M, N;
    void* C;
    int64_t ldc;
    float alpha, beta;
    const float* fa;
    const float* fb;
    const void* bias;
    uint32_t tiles_m, tiles_n, num_tiles, num_kb, group_m;
    uint32_t tma_store;  // C can be stored by TMA, and is not read
};

__device__ __forceinline__ void record_failure(int role, volatile int* abort_flag) {
    atomicCAS(&g_mx_status, 0, role);
    *abort_flag = 1;
}

__device__ __forceinline__ float total_alpha(const MxParams& p) {
    float a = p.alpha;
    if (p.fa != nullptr) a *= __ldg(p.fa);
    if (p.fb != nullptr) a *= __ldg(p.fb);
    return a;
}

template <typename TOut>
__device__ __forceinline__ void put(const MxParams& p, float alpha, int64_t row, int64_t col, float acc) {
    TOut* dst = static_cast<TOut*>(p.C) + row * p.ldc + col;
    const float old = p.beta != 0.0f ? OutT<TOut>::load(dst) : 0.0f;
    const float bv = p.bias != nullptr ? OutT<TOut>::load(static_cast<const TOut*>(p.bias) + col) : 0.0f;
    OutT<TOut>::store(dst, axpby(alpha, acc, p.beta, old) + bv);
}

// ---- the pair kernel -------------------------------------------------------------

constexpr int kPairStages = 5;

template <int kFormat>
struct PairPlan {
    static constexpr int kSf = scale_tiles(kFormat);
    static constexpr uint32_t kA = 128 * kRowBytes;
    static constexpr uint32_t kB = 128 * kRowBytes;
    static constexpr uint32_t kSfa = kSf * kMxTileBytes;
    static constexpr uint32_t kSfb = 2 * kSf * kMxTileBytes;
    static constexpr uint32_t kStage = kA + kB + kSfa + kSfb;
    // epilogue staging: two boxes of 32 rows x 128 bytes per epilogue warp
    static constexpr uint32_t kEpi = kPairStages * kStage;
    static constexpr uint32_t kEpiWarp = 2 * 32 * 128;
    static constexpr uint32_t kBar = kEpi + 4 * kEpiWarp;
    // full[S], scales_full[S], empty[S], scales_ready[2], acc_full[2], acc_free, drain, tmem slot + abort flag
    static constexpr uint32_t kBarBytes = (3 * kPairStages + 6) * 8 + 16;
    static constexpr uint32_t kLaunch = kBar + kBarBytes + 1024;
    // tensor memory: two stages' scales in the last columns, and before them
    // two accumulators of 256 columns that share some (48 with MXFP4's scales,
    // 96 with NVFP4's).  The epilogue reads the shared columns first, after
    // which the next tile's MMAs may start.
    static constexpr uint32_t kSfCols = 12 * kSf;  // 4 for A and 8 for B per scale tile
    static constexpr uint32_t kSfCol = 512 - 2 * kSfCols;
    static constexpr uint32_t kAcc1 = kSfCol - 256;
    static constexpr int kSharedUnits = (256 - kAcc1 + 63) / 64;  // 64-column units that hold them
    static_assert(kStage % 1024 == 0, "stages keep the swizzle atoms aligned");
};

__device__ __forceinline__ void tile_coords(uint32_t t, const MxParams& p, uint32_t& tm, uint32_t& tn) {
    const uint32_t group_size = p.group_m * p.tiles_n;
    const uint32_t group = t / group_size, first_m = group * p.group_m;
    const uint32_t gm = min(p.tiles_m - first_m, p.group_m), r = t % group_size;
    tm = first_m + r % gm;
    tn = r / gm;
}

// A 32 x 64 unit of the tile, lane l its row l, through the staging boxes to C
// by TMA: rows of 128 bytes, 16-byte pieces swizzled so that neither the
// writes nor TMA's reads meet in a bank.  `turn` counts the boxes used.
template <typename TOut>
__device__ __forceinline__ void store_unit(const MxParams& p, const CUtensorMap* tmC, float alpha, uint8_t* boxes, int lane,
                                           int32_t row, int32_t col, const uint32_t (&v)[64], uint32_t& turn) {
    constexpr int kPer = 128 / sizeof(TOut);  // columns of a box
#pragma unroll
    for (int b = 0; b < 64 / kPer; ++b) {
        uint8_t* box = boxes + (turn & 1) * (32 * 128);
        if (lane == 0) bulk_wait_read<1>();  // the store before last has read this box
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(TOut) == 4) {
                    const int c = b * kPer + q * 4 + e;
                    float x = alpha * __uint_as_float(v[c]);
                    if (p.bias != nullptr && col + c < p.N) x += __ldg(static_cast<const float*>(p.bias) + col + c);
                    w[e] = __float_as_uint(x);
                } else {
                    const int c = b * kPer + q * 8 + e * 2;
                    TOut two[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = alpha * __uint_as_float(v[c + h]);
                        if (p.bias != nullptr && col + c + h < p.N)
                            x += OutT<TOut>::load(static_cast<const TOut*>(p.bias) + col + c + h);
                        OutT<TOut>::store(&two[h], x);
                    }
                    memcpy(&w[e], two, 4);
                }
            }
            st_shared_v4(smem_u32(box) + lane * 128 + ((q ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (row < p.M && col + b * kPer < p.N) tma_store_2d(tmC, box, col + b * kPer, row);
            bulk_commit();
        }
        ++turn;
    }
}

// The same where TMA cannot store (C's rows start or end off 16 bytes) or C is read
// (beta): the unit, transposed through the boxes, row by row with a lane on
// columns l and 32 + l.  Element (row, c) lies at word row * 64 + (c + row) % 64,
// so that neither direction meets in a bank.  (8192 x 8192 x 2048 to bf16 with
// an odd leading dimension: 107 us, by TMA into an even one 60 us; 4093 x 4099 x
// 4097 NVFP4 to fp32 47 us.)
template <typename TOut>
__device__ __forceinline__ void store_unit_plain(const MxParams& p, float alpha, uint8_t* boxes, int lane, int64_t row, int64_t col,
                                                 const uint32_t (&v)[64]) {
    const uint32_t words = smem_u32(boxes);
    __syncwarp();  // the last unit's rows have been read
#pragma unroll
    for (int c = 0; c < 64; ++c) st_shared_u32(words + (lane * 64 + ((c + lane) & 63)) * 4, v[c]);
    __syncwarp();
    const bool in0 = col + lane < p.N, in1 = col + 32 + lane < p.N;
    float b0 = 0.0f, b1 = 0.0f;
    if (p.bias != nullptr) {
        const TOut* bias = static_cast<const TOut*>(p.bias) + col + lane;
        if (in0) b0 = OutT<TOut>::load(bias);
        if (in1) b1 = OutT<TOut>::load(bias + 32);
    }
    TOut* dst = static_cast<TOut*>(p.C) + row * p.ldc + col + lane;
    const int rows = static_cast<int>(min(static_cast<int64_t>(32), p.M - row));
    for (int i0 = 0; i0 < rows; i0 += 8) {
        float x[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t line = words + (i0 + i) * 256;
            x[i][0] = ld_shared_f32(line + ((lane + i0 + i) & 63) * 4);
            x[i][1] = ld_shared_f32(line + ((lane + 32 + i0 + i) & 63) * 4);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i, dst += p.ldc) {
            const bool in = i0 + i < rows;
            float old0 = 0.0f, old1 = 0.0f;
            if (p.beta != 0.0f) {
                if (in && in0) old0 = OutT<TOut>::load(dst);
                if (in && in1) old1 = OutT<TOut>::load(dst + 32);
            }
            if (in && in0) OutT<TOut>::store(dst, axpby(alpha, x[i][0], p.beta, old0) + b0);
            if (in && in1) OutT<TOut>::store(dst + 32, axpby(alpha, x[i][1], p.beta, old1) + b1);
        }
    }
}

// Warps: TMA producer, MMA issuer, 4 epilogue, 4 that bring the scales to
// tensor memory (tcgen05.cp would: measured 50 clocks of the tensor pipe per
// 512-byte tile, in line with the MMAs, 72 (MXFP4) to 146 us (NVFP4) of
// 283 to 359 us at 8192^3; tcgen05.st from these warps runs beside them).
constexpr int kPairThreads = 320;

template <int kFormat, typename TOut>
__global__ void __launch_bounds__(kPairThreads, 1)
    mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmSa, const __grid_constant__ CUtensorMap tmSb,
                        const __grid_constant__ CUtensorMap tmC, MxParams p) {
    using S = PairPlan<kFormat>;
    constexpr bool kE8M0 = kFormat == DGA_MXFP4;
    constexpr uint32_t kIdesc0 = idesc_mx(kE8M0, 256, 256, 0), kIdesc2 = idesc_mx(kE8M0, 256, 256, 2);
    constexpr uint16_t kBothCtas = 0x3;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar);
    uint64_t* scales_full = full + kPairStages;
    uint64_t* empty = scales_full + kPairStages;
    uint64_t* scales_ready = empty + kPairStages;
    uint64_t* acc_full = scales_ready + 2;
    uint64_t* acc_free = acc_full + 2;
    uint64_t* drain = acc_free + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&scales_full[s], 1);
            mbar_init(&empty[s], 5);  // the MMAs' commit, one lane of each of this CTA's scale warps
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&scales_ready[b], 8);  // one lane of each scale warp of both CTAs
            mbar_init(&acc_full[b], 1);
        }
        mbar_init(acc_free, 8);  // one lane of each epilogue warp of both CTAs
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmSa);
        tma_prefetch_desc(&tmSb);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t cluster_id = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters) {
                uint32_t tm, tn;
                tile_coords(t, p, tm, tn);
                const int32_t a_row = static_cast<int32_t>(tm * 256 + rank * 128);
                const int32_t b_row = static_cast<int32_t>(tn * 256 + rank * 128);
                for (uint32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleProducer, abort_flag);
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + stage * S::kStage;
                    // the codes of both CTAs count on the leader's barrier, for
                    // its MMA thread; each CTA's scales on its own
                    if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (S::kA + S::kB));
                    mbar_arrive_expect_tx(&scales_full[stage], S::kSfa + S::kSfb);
                    const uint32_t bar = map_to_cta(smem_u32(&full[stage]), 0);
                    const int32_t x = static_cast<int32_t>(kb * kRowBytes);
                    const int32_t sx = static_cast<int32_t>(kb * (S::kSf * kMxTileBytes / 8));
                    tma_load_2d(dst + S::kA + S::kB, &tmSa, &scales_full[stage], sx, a_row / 128);
                    // each CTA's MMA half reads all 256 of the tile's B scales
                    tma_load_2d(dst + S::kA + S::kB + S::kSfa, &tmSb, &scales_full[stage], sx, static_cast<int32_t>(tn * 2));
                    tma_load_2d_pair(dst, &tmA, bar, x, a_row);
                    tma_load_2d_pair(dst + S::kA, &tmB, bar, x, b_row);
                    if (++stage == kPairStages) { stage = 0; phase ^= 1; }
                }
            }
            if (!ok) __nanosleep(20000);  // let copies already issued land before teardown
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            uint32_t stage = 0, phase = 0, i = 0, fill = 0;
            bool ok = true;
            for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters, ++i) {
                if (i > 0 && !mbar_wait_bounded<true>(acc_free, (i - 1) & 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleMma, abort_flag);
                    break;
                }
                const uint32_t d = tmem + (i & 1 ? S::kAcc1 : 0u);
                for (uint32_t kb = 0; kb < p.num_kb; ++kb, ++fill) {
                    if (!mbar_wait_bounded<true>(&full[stage], phase, abort_flag, kWaitLimitNs) ||
                        !mbar_wait_bounded<true>(&scales_ready[fill & 1], (fill >> 1) & 1, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleMma, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = smem_u32(smem + stage * S::kStage);
                    const uint32_t sfa = tmem + S::kSfCol + (fill & 1) * S::kSfCols;
                    const uint32_t sfb = sfa + 4 * S::kSf;
                    const uint64_t a_desc = smem_desc_kmajor_sw128(a_addr);
                    const uint64_t b_desc = smem_desc_kmajor_sw128(a_addr + S::kA);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = kE8M0 ? k / 2 : k;  // the scale tile of these 64 values
                        tc_mma_mx<kE8M0, true>(d, a_desc + 2 * k, b_desc + 2 * k,
                                               kE8M0 && (k & 1) ? kIdesc2 : kIdesc0, sfa + 4 * j, sfb + 8 * j,
                                               (kb > 0 || k > 0) ? 1u : 0u);
                    }
                    tc_commit_pair_multicast(&empty[stage], kBothCtas);
                    if (++stage == kPairStages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit_pair_multicast(&acc_full[i & 1], kBothCtas);
            }
            tc_commit_pair_multicast(drain, 0x1);
            volatile int never = 0;
            mbar_wait_bounded(drain, 0, &never, kWaitLimitNs);
        }
    } else if (warp >= 6) {
        // ------------------------------------------------ scales to tensor memory
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t stage = 0, phase = 0, fill = 0;
        bool ok = true;
        for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters) {
            for (uint32_t kb = 0; kb < p.num_kb; ++kb, ++fill) {
                // the columns are free when the MMAs of two stages ago are done
                const uint32_t before = fill - 2;
                if (!mbar_wait_bounded(&scales_full[stage], phase, abort_flag, kWaitLimitNs) ||
                    (fill >= 2 && !mbar_wait_bounded<true>(&empty[before % kPairStages], (before / kPairStages) & 1,
                                                           abort_flag, kWaitLimitNs))) {
                    record_failure(kRoleScales, abort_flag);
                    ok = false;
                    break;
                }
                // a tile's lane l: the four scales of rows l, 32 + l, 64 + l, 96 + l
                const uint32_t src = smem_u32(smem + stage * S::kStage + S::kA + S::kB) + lane * 16;
                uint32_t r[S::kSfCols];
                auto take = [&](int at, uint32_t from) {
                    const uint4 v = ld_shared_v4(from);
                    r[at] = v.x, r[at + 1] = v.y, r[at + 2] = v.z, r[at + 3] = v.w;
                };
#pragma unroll
                for (int j = 0; j < S::kSf; ++j) {
                    take(4 * j, src + j * kMxTileBytes);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        take(4 * S::kSf + 8 * j + 4 * b, src + S::kSfa + (b * S::kSf + j) * kMxTileBytes);
                }
                tc_fence_after();
                const uint32_t dst = tmem + lane_base + S::kSfCol + (fill & 1) * S::kSfCols;
                if constexpr (S::kSfCols == 24) {
                    tmem_st_32x32b_x16(dst, r);
                    tmem_st_32x32b_x8(dst + 16, r + 16);
                } else {
                    tmem_st_32x32b_x32(dst, r);
                    tmem_st_32x32b_x16(dst + 32, r + 32);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_signal_cluster(map_to_cta(smem_u32(&scales_ready[fill & 1]), 0));
                    // that signal orders tensor memory alone; before TMA writes
                    // the stage's scales anew this warp's reads of them are released
                    mbar_arrive(&empty[stage]);
                }
                if (++stage == kPairStages) { stage = 0; phase ^= 1; }
            }
        }
    } else {
        const int quarter = warp & 3;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* boxes = smem + S::kEpi + (warp - 2) * S::kEpiWarp;
        const float alpha = total_alpha(p);
        uint32_t i = 0, turn = 0;
        for (uint32_t t = cluster_id; t < p.num_tiles; t += n_clusters, ++i) {
            uint32_t tm, tn;
            tile_coords(t, p, tm, tn);
            const int64_t row_base = static_cast<int64_t>(tm) * 256 + rank * 128 + quarter * 32;
            const int64_t col0 = static_cast<int64_t>(tn) * 256;
            if (!mbar_wait_bounded<true>(&acc_full[i & 1], (i >> 1) & 1, abort_flag, kWaitLimitNs)) {
                record_failure(kRoleEpilogue, abort_flag);
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + lane_base + (i & 1 ? S::kAcc1 : 0u);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                // accumulator 0 from its end, 1 from its start: the columns
                // they share are in the first units
                const int unit = i & 1 ? c : 3 - c;
                uint32_t r[64];
                tmem_ld_32x32b_x32(d + unit * 64, reinterpret_cast<uint32_t(&)[32]>(r[0]));
                tmem_ld_32x32b_x32(d + unit * 64 + 32, reinterpret_cast<uint32_t(&)[32]>(r[32]));
                tmem_ld_wait();
                if (c == S::kSharedUnits - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_signal_cluster(map_to_cta(smem_u32(acc_free), 0));
                }
                if (p.tma_store) {
                    store_unit<TOut>(p, &tmC, alpha, boxes, lane, static_cast<int32_t>(row_base),
                                     static_cast<int32_t>(col0) + unit * 64, r, turn);
                } else {
                    store_unit_plain<TOut>(p, alpha, boxes, lane, row_base, col0 + unit * 64, r);
                }
            }
        }
        if (lane == 0) bulk_wait_read<0>();  // shared memory outlives the stores that read it
    }

    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // no CTA frees TMEM or exits while its peer may still touch it
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---- the skinny kernel -------------------------------------------------------------

// kN: rows of A the tile holds (16 to 256).  Two CTAs share an SM where the
// tile is small enough, so that one's start overlaps the other's end.
template <int kFormat, int kN>
struct SkinnyPlan {
    static constexpr int kSf = scale_tiles(kFormat);
    static constexpr int kSfRows = kN > 128 ? 2 : 1;
    static constexpr uint32_t kW = 128 * kRowBytes;
    static constexpr uint32_t kX = kN * kRowBytes;
    static constexpr uint32_t kSw = kSf * kMxTileBytes;
    static constexpr uint32_t kSx = kSfRows * kSf * kMxTileBytes;
    static constexpr uint32_t kStage = kW + kX + kSw + kSx;
    static constexpr int kCtas = kN <= 64 ? 2 : 1;
    static constexpr uint32_t kBudget = (kCtas == 2 ? 110u : 220u) * 1024;
    static constexpr int kStages = kBudget / kStage;
    static constexpr uint32_t kBar = kStages * kStage;
    // full[S], empty[S], acc_full, joined, x_full[S], then tmem slot + abort flag
    static constexpr uint32_t kLaunch = kBar + (3 * kStages + 2) * 8 + 16 + 1024;
    static constexpr uint32_t kSfCol = kN;  // the scales behind the accumulator
    static constexpr uint32_t kUsed = kN + 4 * kSf * (1 + kSfRows);
    static constexpr uint32_t kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
    static_assert(kStage % 1024 == 0, "stages keep the swizzle atoms aligned");
    // K parts: the sums, and those of the other parts, fit the ring
    // (what there is room for: of 256 rows no more parts than two)
    static constexpr uint32_t kMaxSplits = kN > 128 ? 2 : 8;
    static_assert(kBar >= kN * 512 + kN * 512 * (kMaxSplits - 1) / kMaxSplits, "the partial sums fit the ring");
    static_assert(kStages >= 3, "a ring");
};

// A's values, where the kernel quantises them itself.
struct MxSource {
    const void* X;
    int64_t ldx, K;
    int type, vec;  // vec: rows take 16-byte loads
};

// kFused: A comes as values of up to 16 rows and four more warps quantise it,
// a thread 32 values of a stage, while B's codes are under way: one launch, no
// workspace (a token through 4096 x 4096: 6.8 us, as two kernels 8.4 us).
template <int kFormat, int kN, bool kFused, typename TOut>
__global__ void __launch_bounds__(kFused ? 320 : 192, (SkinnyPlan<kFormat, kN>::kCtas))
    mx_gemm_skinny_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                          const __grid_constant__ CUtensorMap tmSw, const __grid_constant__ CUtensorMap tmSx,
                          MxParams p, MxSource src, uint32_t splits) {
    static_assert(!kFused || kN == 16, "a stage of 16 rows is one run of 32 values for each of 128 threads");
    using S = SkinnyPlan<kFormat, kN>;
    constexpr bool kE8M0 = kFormat == DGA_MXFP4;
    constexpr uint32_t kIdesc0 = idesc_mx(kE8M0, 128, kN, 0), kIdesc2 = idesc_mx(kE8M0, 128, kN, 2);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* joined = acc_full + 1;
    uint64_t* x_full = joined + 1;  // kFused: A's codes and scales of a stage
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(x_full + S::kStages);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // the cluster is one tile's K parts
    const uint32_t tile = blockIdx.x / splits, part = blockIdx.x % splits;
    const uint32_t kb0 = part * p.num_kb / splits, kb1 = (part + 1) * p.num_kb / splits;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&x_full[s], 4);  // one lane of each quantising warp
        }
        mbar_init(acc_full, 1);
        mbar_init(joined, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (splits > 1) {
            const int per = kN / static_cast<int>(splits);
            const int mine = max(0, min(per, static_cast<int>(p.M) - static_cast<int>(part) * per));
            if (mine > 0) mbar_arrive_expect_tx(joined, (splits - 1) * mine * 512);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, S::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            const int32_t w_row = static_cast<int32_t>(tile * 128);
            auto load_w = [&](uint32_t stage, uint32_t kb) {
                uint8_t* dst = smem + stage * S::kStage;
                mbar_arrive_expect_tx(&full[stage], kFused ? S::kW + S::kSw : S::kStage);
                tma_load_2d(dst, &tmW, &full[stage], static_cast<int32_t>(kb * kRowBytes), w_row);
                tma_load_2d(dst + S::kW + S::kX, &tmSw, &full[stage], static_cast<int32_t>(kb * (S::kSf * kMxTileBytes / 8)),
                            static_cast<int32_t>(tile));
            };
            auto load_x = [&](uint32_t stage, uint32_t kb) {
                uint8_t* dst = smem + stage * S::kStage;
                tma_load_2d(dst + S::kW, &tmX, &full[stage], static_cast<int32_t>(kb * kRowBytes), 0);
                tma_load_2d(dst + S::kW + S::kX + S::kSw, &tmSx, &full[stage],
                            static_cast<int32_t>(kb * (S::kSf * kMxTileBytes / 8)), 0);
            };
            // a launch right behind the quantisation of A loads B's first
            // stages before it waits: only A is that kernel's output
            const uint32_t first = min(kb1 - kb0, static_cast<uint32_t>(S::kStages));
            for (uint32_t s = 0; s < first; ++s) load_w(s, kb0 + s);
            asm volatile("griddepcontrol.wait;" ::: "memory");
            if (!kFused)
                for (uint32_t s = 0; s < first; ++s) load_x(s, kb0 + s);
            uint32_t stage = 0, phase = 0;
            for (uint32_t kb = kb0 + first; kb < kb1; ++kb) {
                if (!mbar_wait_bounded(&empty[stage], phase, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleProducer, abort_flag);
                    __nanosleep(20000);  // let copies already issued land before teardown
                    break;
                }
                load_w(stage, kb);
                if (!kFused) load_x(stage, kb);
                if (++stage == S::kStages) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs) ||
                    (kFused && !mbar_wait_bounded(&x_full[stage], phase, abort_flag, kWaitLimitNs))) {
                    record_failure(kRoleMma, abort_flag);
                    break;
                }
                tc_fence_after();
                const uint32_t w_addr = smem_u32(smem + stage * S::kStage);
                const uint32_t sf_addr = w_addr + S::kW + S::kX;
                const uint32_t sfw = tmem + S::kSfCol, sfx = sfw + 4 * S::kSf;
#pragma unroll
                for (int j = 0; j < S::kSf; ++j) {
                    tc_cp_scales<false>(sfw + 4 * j, smem_desc_scales(sf_addr + j * kMxTileBytes));
#pragma unroll
                    for (int b = 0; b < S::kSfRows; ++b)
                        tc_cp_scales<false>(sfx + 4 * (S::kSfRows * j + b),
                                            smem_desc_scales(sf_addr + S::kSw + (b * S::kSf + j) * kMxTileBytes));
                }
                const uint64_t w_desc = smem_desc_kmajor_sw128(w_addr);
                const uint64_t x_desc = smem_desc_kmajor_sw128(w_addr + S::kW);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = kE8M0 ? k / 2 : k;
                    tc_mma_mx<kE8M0, false>(tmem, w_desc + 2 * k, x_desc + 2 * k,
                                            kE8M0 && (k & 1) ? kIdesc2 : kIdesc0, sfw + 4 * j,
                                            sfx + 4 * S::kSfRows * j, (kb > kb0 || k > 0) ? 1u : 0u);
                }
                tc_commit(&empty[stage]);
                if (++stage == S::kStages) { stage = 0; phase ^= 1; }
            }
            tc_commit(acc_full);
        }
    }
    __syncwarp();
    if (kFused && warp >= 6) {
        const int row = (warp & 1) * 8 + (lane & 7), run = ((warp - 6) >> 1) * 4 + (lane >> 3);  // of 16 and 8
        const TensorFactor g((kFormat == DGA_NVFP4 && p.fa != nullptr) ? __ldg(p.fa) : 1.0f);
        const int64_t es = src.type == DGA_F32 ? 4 : 2;
        const uint8_t* const X = static_cast<const uint8_t*>(src.X) + row * src.ldx * es;
        uint32_t raw[32] = {};
        auto load = [&](uint32_t kb) {
            const int64_t k = static_cast<int64_t>(kb) * kStageK + run * 32;
            if (row < p.M && kb < kb1) load_run(src.type, X + k * es, src.K - k, src.vec, raw);
        };
        load(kb0);
        uint32_t stage = 0, phase = 0;
        for (uint32_t kb = kb0; kb < kb1; ++kb) {
            uint4 codes;
            uint32_t bytes;
            quantize_run<kFormat>(src.type, raw, g, codes, bytes);
            load(kb + 1);
            if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                record_failure(kRoleScales, abort_flag);
                break;
            }
            uint8_t* x = smem + stage * S::kStage + S::kW;
            st_shared_v4(smem_u32(x) + row * 128 + ((run ^ (row & 7)) << 4), codes);
            uint8_t* scale = x + S::kX + S::kSw + row * 16;  // block b: byte b % 4 of tile b / 4
            if constexpr (kFormat == DGA_MXFP4) scale[(run >> 2) * kMxTileBytes + (run & 3)] = static_cast<uint8_t>(bytes);
            else *reinterpret_cast<uint16_t*>(scale + (run >> 1) * kMxTileBytes + (run & 1) * 2) = static_cast<uint16_t>(bytes);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&x_full[stage]);
            if (++stage == S::kStages) { stage = 0; phase ^= 1; }
        }
        __syncwarp();
    }
    if (warp >= 2 && warp < 6) {
        // Lane: a row of B, that is a column of C; accumulator columns: rows of A
        // ("tokens").  With K in parts, CTA q joins tokens [q per, (q + 1) per).
        // Every CTA puts its sums into the ring, token by token, 128 floats each,
        // and sends each other CTA its tokens by one bulk copy, to a slot of
        // its own behind them; the parts are added up in their order.
        const bool ok = mbar_wait_bounded(acc_full, 0, abort_flag, kWaitLimitNs);
        if (!ok) record_failure(kRoleEpilogue, abort_flag);
        tc_fence_after();
        const int quarter = warp & 3, w = quarter * 32 + lane;
        const int64_t col = static_cast<int64_t>(tile) * 128 + w;
        const int rows = static_cast<int>(p.M), per = kN / static_cast<int>(splits);
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const float alpha = total_alpha(p);
        const float bias = (p.bias != nullptr && col < p.N) ? OutT<TOut>::load(static_cast<const TOut*>(p.bias) + col) : 0.0f;
        TOut* const C = static_cast<TOut*>(p.C) + col;
        auto store = [&](int token, float sum) {
            TOut* dst = C + token * p.ldc;
            const float old = p.beta != 0.0f ? OutT<TOut>::load(dst) : 0.0f;
            OutT<TOut>::store(dst, axpby(alpha, sum, p.beta, old) + bias);
        };
        float* sums = reinterpret_cast<float*>(smem);
        constexpr int kStep = kN < 32 ? 16 : 32;
#pragma unroll 1
        for (int c = 0; c < kN && c < rows; c += kStep) {
            uint32_t r[kStep];
            if constexpr (kStep == 16) tmem_ld_32x32b_x16(tmem + lane_base + c, r);
            else tmem_ld_32x32b_x32(tmem + lane_base + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kStep; ++j) {
                if (splits > 1) sums[(c + j) * 128 + w] = __uint_as_float(r[j]);
                else if (c + j < rows && col < p.N) store(c + j, __uint_as_float(r[j]));
            }
        }
        if (splits > 1) {
            fence_async_shared();
            asm volatile("bar.sync 1, 128;" ::: "memory");  // the four epilogue warps
            cluster_arrive();
            cluster_wait();  // every ring is done with
            const int first = static_cast<int>(part) * per, mine = max(0, min(per, rows - first));
            const float* received = sums + kN * 128;  // part q's slot: q, or q - 1 past this CTA's own
            if (warp == 2 && lane < static_cast<int>(splits) && lane != static_cast<int>(part)) {
                const int theirs = max(0, min(per, rows - lane * per));
                const uint32_t slot = part - (static_cast<int>(part) > lane ? 1 : 0);
                if (theirs > 0)
                    bulk_copy_to_cta(map_to_cta(smem_u32(received + slot * per * 128), lane), smem_u32(sums + lane * per * 128),
                                     theirs * 512, map_to_cta(smem_u32(joined), lane));
            }
            __syncwarp();
            if (mine > 0 && !mbar_wait_bounded<true>(joined, 0, abort_flag, kWaitLimitNs)) record_failure(kRoleEpilogue, abort_flag);
            __syncwarp();
            cluster_arrive_relaxed();  // what was sent here has arrived
            if (col < p.N) {
                // eight tokens at a time: their loads are issued together
                for (int j0 = 0; j0 < mine; j0 += 8) {
                    float sum[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
                    for (int q = 0; q < static_cast<int>(splits); ++q) {
                        const float* src = q == static_cast<int>(part)
                                               ? sums + first * 128
                                               : received + (q - (q > static_cast<int>(part) ? 1 : 0)) * per * 128;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j0 + j < mine) sum[j] += src[(j0 + j) * 128 + w];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j0 + j < mine) store(first + j0 + j, sum[j]);
                }
            }
            __syncwarp();
            cluster_wait();  // and what this CTA sent, at the others
        }
    } else if (splits > 1) {
        cluster_arrive();
        cluster_wait();
        cluster_arrive_relaxed();
        cluster_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmem);
    }
}

// ---- C <- beta C + bias, where there is nothing to multiply -------------------------

template <typename TOut>
__global__ void __launch_bounds__(256) mx_no_product_kernel(MxParams p) {
    const int64_t total = p.M * p.N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256)
        put<TOut>(p, 0.0f, i / p.N, i % p.N, 0.0f);
}

// ---- host side ------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType type, CUtensorMapSwizzle swizzle, const void* base,
                     int64_t inner, int64_t outer, int64_t stride_bytes, uint32_t box_inner, uint32_t box_outer) {
    auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride_bytes)};
    cuuint32_t box[2] = {box_inner, box_outer};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Codes: rows of ceil(K/2) bytes (past them, and past the last row, the copy
// fills zeros: the code of 0).
cudaError_t codes_map(CUtensorMap* map, const MxMatrix& m, int64_t rows, int64_t K, uint32_t box_rows) {
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, m.codes, (K + 1) / 2, rows, m.ld,
                    kRowBytes, box_rows);
}

// Scales: one row of 8-byte words per 128 rows of the matrix.
cudaError_t scales_map(CUtensorMap* map, int format, const MxMatrix& m, int64_t rows, int64_t K, uint32_t box_rows) {
    const int64_t tiles_k = mx_tiles_k(format, K);
    return make_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, CU_TENSOR_MAP_SWIZZLE_NONE, m.scales,
                    tiles_k * (kMxTileBytes / 8), (rows + 127) / 128, tiles_k * kMxTileBytes,
                    static_cast<uint32_t>(scale_tiles(format) * kMxTileBytes / 8), box_rows);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), unsigned grid, int threads, unsigned cluster, int smem, bool pdl,
                   cudaStream_t s, const A&... args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <int kFormat, int kN, bool kFused, typename TOut>
cudaError_t launch_skinny(const MxGemmArgs& a, MxParams p, const DeviceInfo& dev) {
    using S = SkinnyPlan<kFormat, kN>;
    CUtensorMap m[4];
    cudaError_t e = codes_map(&m[0], a.B, a.N, a.K, 128);
    if (e == cudaSuccess) e = scales_map(&m[2], kFormat, a.B, a.N, a.K, 1);
    if (kFused) {
        m[1] = m[0], m[3] = m[2];  // not used
    } else {
        if (e == cudaSuccess) e = codes_map(&m[1], a.A, a.M, a.K, kN);
        if (e == cudaSuccess) e = scales_map(&m[3], kFormat, a.A, a.M, a.K, S::kSfRows);
    }
    if (e != cudaSuccess) return e;
    const MxSource src{a.X, a.ldx, a.K, a.x_dtype, aligned(a.X, 16) && a.ldx % (a.x_dtype == DGA_F32 ? 4 : 8) == 0};
    // parts of K: as many as fill the machine's CTA slots, each at least two stages
    const int64_t tiles = (a.N + 127) / 128, slots = static_cast<int64_t>(dev.sm_count) * S::kCtas;
    uint32_t splits = 1;
    while (splits < S::kMaxSplits && tiles * splits * 2 <= slots && p.num_kb >= splits * 4) splits *= 2;
    return launch(mx_gemm_skinny_kernel<kFormat, kN, kFused, TOut>, static_cast<unsigned>(tiles * splits), kFused ? 320 : 192,
                  splits, static_cast<int>(S::kLaunch), a.after_quantize, a.stream, m[0], m[1], m[2], m[3], p, src, splits);
}

template <int kFormat, typename TOut>
cudaError_t launch_pair(const MxGemmArgs& a, MxParams p, const DeviceInfo& dev) {
    using S = PairPlan<kFormat>;
    CUtensorMap m[5];
    cudaError_t e = codes_map(&m[0], a.A, a.M, a.K, 128);
    if (e == cudaSuccess) e = codes_map(&m[1], a.B, a.N, a.K, 128);
    if (e == cudaSuccess) e = scales_map(&m[2], kFormat, a.A, a.M, a.K, 1);
    if (e == cudaSuccess) e = scales_map(&m[3], kFormat, a.B, a.N, a.K, 2);
    if (e != cudaSuccess) return e;
    p.tiles_m = static_cast<uint32_t>((a.M + 255) / 256);
    p.tiles_n = static_cast<uint32_t>((a.N + 255) / 256);
    p.num_tiles = p.tiles_m * p.tiles_n;
    // tile rows walked together: their A panels stay in L2 while B passes
    const double panel = 256.0 * static_cast<double>(a.K) / 2;
    p.group_m = std::min(p.tiles_m, std::max(8u, std::min(64u, static_cast<uint32_t>(32.0 * 1024 * 1024 / panel))));
    const unsigned clusters = std::min<unsigned>(p.num_tiles, dev.sm_count / 2);
    // C by TMA stores where it is only written and its rows start and end on 16
    // bytes: TMA writes the whole 16 bytes that a row's end lies in
    constexpr int64_t kEs = sizeof(TOut);
    p.tma_store = a.beta == 0.0f && aligned(a.C, 16) && a.ldc * kEs % 16 == 0 && a.N * kEs % 16 == 0;
    if (p.tma_store)
        e = make_map(&m[4], kEs == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                     CU_TENSOR_MAP_SWIZZLE_128B, a.C, a.N, a.M, a.ldc * kEs, 128 / kEs, 32);
    else
        m[4] = m[0];  // not used
    if (e != cudaSuccess) return e;
    // (it waits for the grid before it ahead of its first load)
    return launch(mx_gemm_pair_kernel<kFormat, TOut>, 2 * clusters, kPairThreads, 2, static_cast<int>(S::kLaunch), true,
                  a.stream, m[0], m[1], m[2], m[3], m[4], p);
}

template <int kFormat, typename TOut>
cudaError_t launch_as(const MxGemmArgs& a, const DeviceInfo& dev) {
    MxParams p{};
    p.M = a.M;
    p.N = a.N;
    p.C = a.C;
    p.ldc = a.ldc;
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.fa = a.A.factor;
    p.fb = a.B.factor;
    p.bias = a.bias;
    if (a.K == 0 || a.alpha == 0.0f) {
        const int64_t blocks = std::min<int64_t>((a.M * a.N + 255) / 256, static_cast<int64_t>(dev.sm_count) * 16);
        mx_no_product_kernel<TOut><<<static_cast<unsigned>(blocks), 256, 0, a.stream>>>(p);
        return cudaGetLastError();
    }
    p.num_kb = static_cast<uint32_t>((a.K + kStageK - 1) / kStageK);
    if (a.X != nullptr) return launch_skinny<kFormat, 16, true, TOut>(a, p, dev);
    if (a.M <= 16) return launch_skinny<kFormat, 16, false, TOut>(a, p, dev);
    if (a.M <= 32) return launch_skinny<kFormat, 32, false, TOut>(a, p, dev);
    if (a.M <= 64) return launch_skinny<kFormat, 64, false, TOut>(a, p, dev);
    if (a.M <= 128) return launch_skinny<kFormat, 128, false, TOut>(a, p, dev);
    if (a.M <= 256) return launch_skinny<kFormat, 256, false, TOut>(a, p, dev);
    return launch_pair<kFormat, TOut>(a, p, dev);
}

}  // namespace

cudaError_t mx_gemm_launch(const MxGemmArgs& a, const DeviceInfo& dev, int* launches) {
    cudaError_t e;
    const bool mx = a.format == DGA_MXFP4;
    switch (a.out_dtype) {
    case DGA_F32: e = mx ? launch_as<DGA_MXFP4, float>(a, dev) : launch_as<DGA_NVFP4, float>(a, dev); break;
    case DGA_BF16: e = mx ? launch_as<DGA_MXFP4, __nv_bfloat16>(a, dev) : launch_as<DGA_NVFP4, __nv_bfloat16>(a, dev); break;
    default: e = mx ? launch_as<DGA_MXFP4, __half>(a, dev) : launch_as<DGA_NVFP4, __half>(a, dev); break;
    }
    if (e == cudaSuccess) ++*launches;
    return e;
}

cudaError_t mx_status_take(int* status) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_mx_status, sizeof v);
    if (e != cudaSuccess) return e;
    if (v != 0) {
        int zero = 0;
        e = cudaMemcpyToSymbol(g_mx_status, &zero, sizeof zero);
    }
    *status = v;
    return e;
}

}  // namespace dga
