// q4_rows.cuh -- products of a few rows (up to 64) with a 4-bit weight with group scales,
//     Y[M, N] = X[M, K] ((q - z) s)[N, K]^T + bias,
// and the gated layer H = act(g) * u on them.
//
// The bytes of the codes are its floor (half a byte to a weight), so each is read
// once and multiplied as what it is: q - z is a small integer, exact in bf16 and
// fp16, and mma.sync m16n8k16 multiplies it by X exactly and sums in fp32; the
// sum over (a part of) a group is then scaled by s in fp32.  No weight is rounded.
// 8192 x 8192 in groups of 128, bf16, one row: 14.4 us where the bytes take 5.2; no pipe is
// full (ALU 57 %, issue 52 %, DRAM 25 %): eleven steps to eight codes, and the scales' table,
// which is filled before the first of them.
//
//  * The grid is whole waves of a block per SM, and the weight's rows are shared
//    out evenly, up to 64 to a block (of a gated layer up to 32 gate rows and the
//    up rows that go with them).
//  * A ring of stages in shared memory: a producer thread brings the rows' codes
//    (boxes of 256 columns, 128-byte swizzle) and X's values by TMA, so that what
//    is in flight does not take registers.  The scales and zero points of the
//    block's rows, over all of K, are put into shared memory at the start.
//  * Sixteen consumer warps (eight for more than 16 rows) share the stage's columns, 64 at a time, and the
//    tiles of 16 weight rows.  The
//    weight is the MMA's A, X its B.  Which k an MMA's columns stand for is free
//    as long as A and B agree, so a lane reads consecutive codes of its rows: 16
//    of 64, or 8 of each 32 where the groups are that small.
//  * A word of 8 codes becomes four registers of two: (w >> 4 i) & 0x000f000f
//    has codes i and i + 4, and or-ed into the mantissa of 128 (bf16) or 1024
//    (fp16) they are 128 + q or 1024 + q; subtracting 128 + z or 1024 + z is
//    exact.  X's eight values are paired alike.  bf16's range is fp32's, so there the
//    same fused step takes 2^-10 of the difference, which 64 columns of the largest
//    values and codes cannot overflow; the sums regain it at the end (both exact).
//  * The warps' sums meet in shared memory and are added in a fixed order; bias,
//    activation and product follow from there.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "gated_act.cuh"
#include "mx_common.cuh"
#include "ptx.cuh"

namespace dga {

namespace q4rows {

// non-zero: a bounded wait expired (role code); one for each file's kernels
static __device__ int g_status;

// Reads and clears this file's word of the current device.
static cudaError_t take_status(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_status, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_status, &zero, sizeof zero);
    *status = v;
    return e;
}

constexpr int kMaxStages = 8;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr uint32_t kBarBytes = 2 * kMaxStages * 8 + 16;
constexpr uint32_t kMostSmem = 226 * 1024;
constexpr uint32_t kMostTable = 100 * 1024;  // scales and zero points in shared memory, else read from memory
enum : int { kRoleProducer = 1, kRoleConsumer = 2 };

struct Params {
    int64_t M, N, K;  // N: outputs (a gated layer's F)
    Q4Matrix q;
    const void* bias;
    void* Y;
    int64_t ldy;
    int act, gated;
    int shift;           // log2 of the group
    uint32_t box_rows;   // most rows of a block (gated: of each half)
    uint32_t n_stages_k, stages, stage_bytes, ring_bytes;
    uint32_t table_pitch;  // entries between rows of the table, 0: none
    int table_vec;         // eight scales (zero points) take one aligned load
    uint32_t chunk_inverse;  // ceil(2^32 / (table_pitch / 8)), 0 for one chunk to a row
};

template <int kMt>
struct Plan {
    // consumer warps: sixteen where the registers allow
    static constexpr int kConsumers = kMt <= 2 ? 16 : 8, kThreads = (kConsumers + 1) * 32;
    static constexpr int kStageK = kMt == 8 ? 256 : kMt == 1 ? 1024 : 512;
    static constexpr int kBoxes = kStageK / 256, kUnits = kStageK / 64;
    // tiles of a block a warp has, so that its sums fit the registers
    __host__ __device__ static constexpr int per_warp(int tiles) { return kMt == 1 ? tiles : kMt == 8 || tiles == 1 ? 1 : tiles / 2; }
};

inline uint32_t stage_columns(int64_t M) {
    return M <= 8 ? Plan<1>::kStageK : M <= 16 ? Plan<2>::kStageK : M <= 32 ? Plan<4>::kStageK : Plan<8>::kStageK;
}

template <typename T> struct Codes;
template <> struct Codes<__nv_bfloat16> {
    static constexpr uint32_t kBoth = 0x43004300u;  // 128
    static constexpr uint32_t kBase = 0xbe00u;      // -128 / 1024, its last place 1 / 1024
    static constexpr float kUnit = 1024.0f;         // what the sums are to be multiplied by
    // a / 1024 + b
    __device__ __forceinline__ static uint32_t less(uint32_t a, uint32_t b) {
        const uint32_t factors = 0x3a803a80u;  // 1 / 1024
        __nv_bfloat162 x, y, f;
        memcpy(&x, &a, 4);
        memcpy(&y, &b, 4);
        memcpy(&f, &factors, 4);
        x = __hfma2(x, f, y);
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ __forceinline__ static float scale(uint32_t entry) { return __uint_as_float(entry & 0xffff0000u); }
    // (q - z) / kUnit of a word's codes 0 and 4, 1 and 5, 2 and 6, 3 and 7; z: the base twice.
    __device__ __forceinline__ static void unpack(uint32_t (&c)[4], uint32_t w, uint32_t z) {
        c[0] = less((w & 0x000f000fu) | kBoth, z);
        c[1] = less(((w >> 4) & 0x000f000fu) | kBoth, z);
        c[2] = less(((w >> 8) & 0x000f000fu) | kBoth, z);
        c[3] = less(((w >> 12) & 0x000f000fu) | kBoth, z);
    }
    // d = a b + (first ? 0 : d)
    __device__ __forceinline__ static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
        if (first) {
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        } else {
            asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        }
    }
};
template <> struct Codes<__half> {
    static constexpr uint32_t kBase = 0x6400u, kBoth = 0x64006400u;  // 1024
    static constexpr float kUnit = 1.0f;
    __device__ __forceinline__ static uint32_t minus(uint32_t a, uint32_t b) {
        __half2 x, y;
        memcpy(&x, &a, 4);
        memcpy(&y, &b, 4);
        x = __hsub2(x, y);
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    // The same; a byte's upper code stands as 1024 + 16 q, which a sixteenth, less 64 + z,
    // is in one fused step.
    __device__ __forceinline__ static void unpack(uint32_t (&c)[4], uint32_t w, uint32_t z) {
        const uint32_t v = w >> 8, z64 = minus(0x63806380u, z);  // 960 - (1024 + z)
        c[0] = minus((w & 0x000f000fu) | kBoth, z);
        c[1] = sixteenth((w & 0x00f000f0u) | kBoth, z64);
        c[2] = minus((v & 0x000f000fu) | kBoth, z);
        c[3] = sixteenth((v & 0x00f000f0u) | kBoth, z64);
    }
    __device__ __forceinline__ static uint32_t sixteenth(uint32_t a, uint32_t z64) {
        __half2 x, y;
        memcpy(&x, &a, 4);
        memcpy(&y, &z64, 4);
        x = __hfma2(x, __float2half2_rn(0.0625f), y);
        uint32_t r;
        memcpy(&r, &x, 4);
        return r;
    }
    __device__ __forceinline__ static float scale(uint32_t entry) { return __half2float(__ushort_as_half(static_cast<unsigned short>(entry >> 16))); }
    // d = a b + (first ? 0 : d)
    __device__ __forceinline__ static void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
        if (first) {
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
        } else {
            asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
        }
    }
};

__device__ __forceinline__ void record_failure(int role, volatile int* abort_flag) {
    atomicCAS(&g_status, 0, role);
    *abort_flag = 1;
}

// A group's scale and base (fp16: 1024 plus the zero point, bf16: -1/1024 of 128 plus it) as the table holds
// them: for groups of 32 one word, the scale's bits above the base's, else two,
// the scale in fp32 and the base twice.
template <bool kSmall> struct EntryOf { using type = uint2; };
template <> struct EntryOf<true> { using type = uint32_t; };

template <typename T, bool kSmall>
__device__ __forceinline__ typename EntryOf<kSmall>::type make_entry(uint32_t scale, uint32_t zero) {
    const uint32_t word = (scale << 16) | (Codes<T>::kBase + (zero & 15u));
    if constexpr (kSmall) return word;
    else return make_uint2(__float_as_uint(Codes<T>::scale(word)), __byte_perm(word, 0, 0x1010));
}

// The same from memory; 0 past the block's rows or the groups.
template <typename T, bool kSmall>
__device__ __forceinline__ typename EntryOf<kSmall>::type read_entry(const Params& p, int64_t row, int64_t group, int64_t groups, bool in) {
    if (!in || group >= groups) return make_entry<T, kSmall>(0, 0);
    return make_entry<T, kSmall>(__ldg(static_cast<const uint16_t*>(p.q.scales) + row * p.q.ld_scales + group),
                                 p.q.zeros ? __ldg(p.q.zeros + row * p.q.ld_zeros + group) : 8u);
}

// The table of a block's rows: eight groups to a thread at a time, four of them
// in flight (one group at a time, each behind the last one's loads, took longer
// than the product: 16 of 24 us at 8192 x 8192).
template <typename T, bool kSmall, int kRows, int kConsumers>
__device__ __forceinline__ void fill_table(const Params& p, typename EntryOf<kSmall>::type* table, int64_t n0, int count, int half_rows, int64_t groups) {
    constexpr int kAhead = 4;
    const uint32_t chunks = (p.table_pitch - 1) / 8, total = kRows * chunks;
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += kAhead * kConsumers * 32) {
        uint4 s[kAhead];
        uint2 z[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t e = e0 + u * kConsumers * 32, r = p.chunk_inverse ? __umulhi(e, p.chunk_inverse) : e;
            const int64_t group = (e - r * chunks) * 8;
            const int at = static_cast<int>(r) >= half_rows ? static_cast<int>(r) - half_rows : static_cast<int>(r);
            const int64_t row = n0 + at + (static_cast<int>(r) >= half_rows ? p.N : 0);
            s[u] = make_uint4(0, 0, 0, 0);
            z[u] = p.q.zeros ? make_uint2(0, 0) : make_uint2(0x08080808u, 0x08080808u);
            if (e >= total || at >= count || group >= groups) continue;
            const uint16_t* sp = static_cast<const uint16_t*>(p.q.scales) + row * p.q.ld_scales + group;
            const uint8_t* zp = p.q.zeros + row * p.q.ld_zeros + group;
            if (p.table_vec && group + 8 <= groups) {
                s[u] = __ldg(reinterpret_cast<const uint4*>(sp));
                if (p.q.zeros) z[u] = __ldg(reinterpret_cast<const uint2*>(zp));
            } else {
                uint32_t sw[4] = {0, 0, 0, 0}, zw[2] = {z[u].x, z[u].y};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (group + i >= groups) break;
                    sw[i / 2] |= static_cast<uint32_t>(__ldg(sp + i)) << (16 * (i & 1));
                    if (p.q.zeros) zw[i / 4] |= static_cast<uint32_t>(__ldg(zp + i)) << (8 * (i & 3));
                }
                s[u] = make_uint4(sw[0], sw[1], sw[2], sw[3]);
                z[u] = make_uint2(zw[0], zw[1]);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint32_t e = e0 + u * kConsumers * 32, r = p.chunk_inverse ? __umulhi(e, p.chunk_inverse) : e;
            if (e >= total) break;
            auto* dst = table + r * p.table_pitch + (e - r * chunks) * 8;
            const uint32_t sw[4] = {s[u].x, s[u].y, s[u].z, s[u].w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                dst[i] = make_entry<T, kSmall>((sw[i / 2] >> (16 * (i & 1))) & 0xffffu, (i < 4 ? z[u].x : z[u].y) >> (8 * (i & 3)));
        }
    }
}

// kTiles: tiles of 16 weight rows to a block; kMt: tiles of 8 rows of X;
// kSmall: groups of 32 (else 64 or 128).
template <typename T, bool kSmall, int kMt, int kTiles>
__global__ void __launch_bounds__(Plan<kMt>::kThreads, 1) q4_rows_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tmX,
               const __grid_constant__ CUtensorMap tmTail, Params p) {
    using S = Plan<kMt>;
    constexpr int kConsumers = S::kConsumers;
    constexpr int kPer = S::per_warp(kTiles), kTileGroups = kTiles / kPer, kParts = kConsumers / kTileGroups < S::kUnits ? kConsumers / kTileGroups : S::kUnits;
    constexpr uint32_t kCodeBytes = S::kBoxes * kTiles * 2048;
    constexpr int kRows = kTiles * 16, kPitch = kRows + 4;

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // known to be shared memory
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.ring_bytes);
    uint64_t* empty = full + kMaxStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kMaxStages);
    using Entry = typename EntryOf<kSmall>::type;
    Entry* table = reinterpret_cast<Entry*>(smem + p.ring_bytes + kBarBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * p.N / gridDim.x;
    const int count = static_cast<int>((static_cast<int64_t>(blockIdx.x) + 1) * p.N / gridDim.x - n0);
    const int half_rows = p.gated ? kRows / 2 : kRows;  // up rows follow from here
    const int64_t groups = (p.K + (1 << p.shift) - 1) >> p.shift;
    const uint32_t x_rows = static_cast<uint32_t>(p.M);

    if (threadIdx.x == kConsumers * 32) {
        tma_prefetch_desc(&tm);
        if (p.K >= S::kStageK) tma_prefetch_desc(&tmX);
        if (p.K % S::kStageK) tma_prefetch_desc(&tmTail);
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kConsumers);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == kConsumers) {
        // ------------------------------------------------ copies
        if (lane == 0) {
            const uint32_t bytes = S::kBoxes * p.box_rows * 128 * (p.gated ? 2 : 1) + S::kUnits * x_rows * 128;
            uint32_t stage = 0, phase = 0;
            for (uint32_t i = 0; i < p.n_stages_k; ++i) {
                if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleProducer, abort_flag);
                    __nanosleep(20000);  // let copies already issued land before teardown
                    break;
                }
                uint8_t* dst = smem + stage * p.stage_bytes;
                mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
                for (int b = 0; b < S::kBoxes; ++b) {
                    const int32_t x = static_cast<int32_t>((i * S::kBoxes + b) * 128);
                    tma_load_2d(dst + b * kTiles * 2048, &tm, &full[stage], x, static_cast<int32_t>(n0));
                    if (p.gated)
                        tma_load_2d(dst + b * kTiles * 2048 + kTiles * 1024, &tm, &full[stage], x, static_cast<int32_t>(n0 + p.N));
                }
                // X as [64 columns][M rows]: a stage in one copy, the one that K ends in by as
                // many as it has (a copy takes some 75 clocks whatever its size)
                if (static_cast<int64_t>(i + 1) * S::kStageK <= p.K) {
                    tma_load_3d(dst + kCodeBytes, &tmX, &full[stage], 0, 0, static_cast<int32_t>(i * S::kUnits));
                } else {
                    for (int u = 0; u < S::kUnits; ++u)
                        tma_load_2d(dst + kCodeBytes + u * x_rows * 128, &tmTail, &full[stage], static_cast<int32_t>((i * S::kUnits + u) * 64), 0);
                }
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
        }
        return;
    }

    // ---------------------------------------------------- consumers
    if (p.table_pitch) {
        fill_table<T, kSmall, kRows, kConsumers>(p, table, n0, count, half_rows, groups);
        asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    }
    const int g = lane >> 2, t = lane & 3;
    // which row of 8 a lane has, and which row of X the lane's column is: the orders
    // that keep the reads below free of bank conflicts
    const int row8 = kSmall ? g : ((g & 3) << 1) | (g >> 2);
    const int token8 = kSmall ? ((g & 1) << 2) | (g >> 1) : g;
    const int part = warp % kParts, tile0 = warp / kParts * kPer;
    const bool idle = tile0 >= kTiles;  // fewer units of work than warps
    const uint32_t code_lane = tile0 * 2048 + row8 * 128;
    const Entry* table_lane = table + (tile0 * 16 + row8) * p.table_pitch;
    // X's lines of 128 bytes in a stage: of a unit, of a tile of 8 rows.  A lane whose
    // row there is past M reads the last one's: its column of the sums is not used
    int x_row[kMt];
#pragma unroll
    for (int m = 0; m < kMt; ++m) x_row[m] = min(m * 8 + token8, static_cast<int>(x_rows) - 1);

    float acc[kPer][kMt][4];
#pragma unroll
    for (int r = 0; r < kPer; ++r)
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][m][i] = 0.0f;

    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (uint32_t i = 0; i < p.n_stages_k; ++i) {
        if (!mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs)) {
            if (lane == 0) record_failure(kRoleConsumer, abort_flag);
            ok = false;
            break;
        }
        const uint8_t* base = smem + stage * p.stage_bytes;
#pragma unroll
        for (int v = 0; v < S::kUnits / kParts; ++v) {
            if (idle) break;
            const int unit = v * kParts + part;  // 64 columns
            const uint8_t* codes = base + code_lane + (unit >> 2) * (kTiles * 2048);
            uint32_t w[kPer][2][2];
#pragma unroll
            for (int r = 0; r < kPer; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* at = codes + r * 2048 + h * 1024;
                    if constexpr (kSmall) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) w[r][h][e] = *reinterpret_cast<const uint32_t*>(at + ((((unit & 3) * 2 + e) ^ row8) << 4) + t * 4);
                    } else {
                        const uint2 two = *reinterpret_cast<const uint2*>(at + ((((unit & 3) * 2 + (t >> 1)) ^ row8) << 4) + (t & 1) * 8);
                        w[r][h][0] = two.x, w[r][h][1] = two.y;
                    }
                }
            constexpr int kScales = kSmall ? 2 : 1;
            Entry entry[kPer][2][kScales];
            const uint32_t group = (i * S::kStageK + unit * 64) >> p.shift;
#pragma unroll
            for (int r = 0; r < kPer; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < kScales; ++e) {
                        if (p.table_pitch) {
                            entry[r][h][e] = table_lane[(r * 16 + h * 8) * p.table_pitch + group + e];
                        } else {
                            const int row = (tile0 + r) * 16 + h * 8 + row8, at = row >= half_rows ? row - half_rows : row;
                            entry[r][h][e] = read_entry<T, kSmall>(p, n0 + at + (row >= half_rows ? p.N : 0), group + e, groups, at < count);
                        }
                    }
            float sum[kPer][kMt][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t b[kMt][4];
#pragma unroll
                for (int m = 0; m < kMt; ++m) {
                    const uint32_t line = unit * x_rows + x_row[m];
                    const uint4 x = *reinterpret_cast<const uint4*>(base + kCodeBytes + line * 128 + (((kSmall ? 4 * e + t : 2 * t + e) ^ (line & 7)) << 4));
                    b[m][0] = __byte_perm(x.x, x.z, 0x5410);  // values 0 and 4
                    b[m][1] = __byte_perm(x.x, x.z, 0x7632);  // 1 and 5
                    b[m][2] = __byte_perm(x.y, x.w, 0x5410);  // 2 and 6
                    b[m][3] = __byte_perm(x.y, x.w, 0x7632);  // 3 and 7
                }
#pragma unroll
                for (int r = 0; r < kPer; ++r) {
                    const bool first = kSmall || e == 0;  // of the group's part
                    uint32_t z[2];
                    float scale[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if constexpr (kSmall) {
                            z[h] = __byte_perm(entry[r][h][e], 0, 0x1010);
                            scale[h] = Codes<T>::scale(entry[r][h][e]);
                        } else {
                            z[h] = entry[r][h][0].y;
                            scale[h] = __uint_as_float(entry[r][h][0].x);
                        }
                    }
                    uint32_t c[2][4];
                    Codes<T>::unpack(c[0], w[r][0][e], z[0]);
                    Codes<T>::unpack(c[1], w[r][1][e], z[1]);
                    const uint32_t a0[4] = {c[0][0], c[1][0], c[0][1], c[1][1]}, a1[4] = {c[0][2], c[1][2], c[0][3], c[1][3]};
#pragma unroll
                    for (int m = 0; m < kMt; ++m) {
                        Codes<T>::mma(sum[r][m], a0, b[m][0], b[m][1], first);
                        Codes<T>::mma(sum[r][m], a1, b[m][2], b[m][3], false);
                    }
                    if (kSmall || e == 1) {
#pragma unroll
                        for (int m = 0; m < kMt; ++m) {
                            acc[r][m][0] = fmaf(scale[0], sum[r][m][0], acc[r][m][0]);
                            acc[r][m][1] = fmaf(scale[0], sum[r][m][1], acc[r][m][1]);
                            acc[r][m][2] = fmaf(scale[1], sum[r][m][2], acc[r][m][2]);
                            acc[r][m][3] = fmaf(scale[1], sum[r][m][3], acc[r][m][3]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == p.stages) { stage = 0; phase ^= 1; }
    }

    // every copy has landed and every warp has read the ring: the sums take its place
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    if (*abort_flag) ok = false;
    float* sums = reinterpret_cast<float*>(smem);  // [part][8 kMt][kPitch]
#pragma unroll
    for (int r = 0; r < kPer && !idle; ++r)
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int col = 2 * t + (j & 1);
                const int token = m * 8 + (kSmall ? ((col & 1) << 2) | (col >> 1) : col);
                sums[(part * 8 * kMt + token) * kPitch + (tile0 + r) * 16 + row8 + 8 * (j >> 1)] = acc[r][m][j];
            }
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    if (!ok) return;
    const T* bias = static_cast<const T*>(p.bias);
    const int outputs = static_cast<int>(p.M) * half_rows;
    for (int o = threadIdx.x; o < outputs; o += kConsumers * 32) {
        const int token = o / half_rows, c = o % half_rows;
        if (c >= count) continue;
        const int64_t n = n0 + c;
        auto total = [&](int col) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kParts; ++k) v += sums[(k * 8 * kMt + token) * kPitch + col];
            return v * Codes<T>::kUnit;
        };
        float v = total(c);
        if (bias) v += OutT<T>::load(bias + n);
        if (p.gated) {
            float u = total(half_rows + c);
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
        OutT<T>::store(static_cast<T*>(p.Y) + token * p.ldy + n, v);
    }
}

template <typename T, bool kSmall, int kMt, int kTiles>
cudaError_t launch(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, Params p, unsigned blocks, cudaStream_t s) {
    using S = Plan<kMt>;
    constexpr int kConsumers = S::kConsumers;
    auto kern = q4_rows_kernel<T, kSmall, kMt, kTiles>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostSmem));
    if (e != cudaSuccess) return e;
    p.n_stages_k = static_cast<uint32_t>((p.K + S::kStageK - 1) / S::kStageK);
    const uint64_t n = ((static_cast<uint64_t>(p.n_stages_k) * S::kStageK >> p.shift) + 7) / 8 * 8;
    // an odd number of entries between the rows of the table: no two of 8 meet in a bank
    const uint64_t table = (n + 1) * kTiles * 16 * sizeof(typename EntryOf<kSmall>::type);
    p.table_pitch = table <= kMostTable ? static_cast<uint32_t>(n + 1) : 0;
    const uint32_t fixed = kBarBytes + 1024 + (p.table_pitch ? static_cast<uint32_t>(table) : 0);
    const uint64_t chunks = n / 8;  // to a row; exact below 2^32 / chunks entries
    p.chunk_inverse = chunks > 1 ? static_cast<uint32_t>(((uint64_t{1} << 32) + chunks - 1) / chunks) : 0;
    p.stage_bytes = S::kBoxes * kTiles * 2048 + (S::kUnits * static_cast<uint32_t>(p.M) * 128 + 1023) / 1024 * 1024;
    p.stages = std::min<uint32_t>({static_cast<uint32_t>(kMaxStages), (kMostSmem - fixed) / p.stage_bytes, p.n_stages_k});
    static_assert((kMostSmem - kBarBytes - 1024 - kMostTable) / (S::kBoxes * kTiles * 2048 + S::kUnits * kMt * 1024) >= 2, "two stages at least");
    // the warps' sums take the ring's place
    constexpr int kMostParts = kConsumers / (kTiles / S::per_warp(kTiles));
    constexpr uint32_t kSums = (kMostParts < S::kUnits ? kMostParts : S::kUnits) * 8 * kMt * (kTiles * 16 + 4) * 4;
    static_assert(kSums + kBarBytes + 1024 + kMostTable <= kMostSmem, "they fit");
    p.ring_bytes = std::max(p.stages * p.stage_bytes, (kSums + 1023) / 1024 * 1024);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = p.ring_bytes + fixed;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tm, tmX, tmTail, p);
}

template <typename T, bool kSmall, int kMt>
cudaError_t launch_tiles(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s) {
    return tiles == 1 ? launch<T, kSmall, kMt, 1>(tm, tmX, tmTail, p, blocks, s)
           : tiles == 2 ? launch<T, kSmall, kMt, 2>(tm, tmX, tmTail, p, blocks, s) : launch<T, kSmall, kMt, 4>(tm, tmX, tmTail, p, blocks, s);
}

template <typename T, bool kSmall>
cudaError_t launch_mt(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s) {
    return p.M <= 8 ? launch_tiles<T, kSmall, 1>(tm, tmX, tmTail, p, tiles, blocks, s)
           : p.M <= 16 ? launch_tiles<T, kSmall, 2>(tm, tmX, tmTail, p, tiles, blocks, s)
           : p.M <= 32 ? launch_tiles<T, kSmall, 4>(tm, tmX, tmTail, p, tiles, blocks, s) : launch_tiles<T, kSmall, 8>(tm, tmX, tmTail, p, tiles, blocks, s);
}

template <typename T>
cudaError_t launch_type(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s) {
    return p.q.group == 32 ? launch_mt<T, true>(tm, tmX, tmTail, p, tiles, blocks, s) : launch_mt<T, false>(tm, tmX, tmTail, p, tiles, blocks, s);
}

cudaError_t launch_bf16(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s);
cudaError_t launch_f16(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s);
cudaError_t take_status_f16(int* status);

}  // namespace q4rows
}  // namespace dga
