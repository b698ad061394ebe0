// newton_schulz.cu -- an update's orthogonalisation by Newton-Schulz products.
//
// G (one matrix or a batch) is scaled to X = G / (|G|_F + eps), transposed
// where it has more rows than columns (m <= n from here on), and each step
// replaces X by an odd quintic of it,
//
//     A = X X^T,   B = b A + c A^2,   X <- a X + B X,
//
// which drives every singular value of X towards 1: the iteration of K.
// Jordan, "Muon: An optimizer for hidden layers in neural networks" (2024).
// A step costs m^2 n + m^3 + 2 m^2 n operations when the symmetric A and B
// are formed by their upper triangle alone, as they are here.
//
// Numbers.  X, A and B live in the workspace as fp16, times 2^12 (their
// entries stay far below 16 in magnitude, and what is small keeps its
// digits), and are multiplied by tcgen05 with fp32 accumulation.
//   * X is held as the sum of two fp16 numbers, hi + lo: 22 bits.  A one-word
//     X would round every step's a X, an error in all directions, which the
//     following steps amplify by up to a per step where X's singular values
//     are small (simulated: 1e-2 to 4e-2 off for momentum of low rank).
//   * bf16 output: the products take hi alone.  Their roundings multiply A, B
//     or X by 1 + O(2^-12) on either side and so stay within X's own singular
//     subspaces: 1e-4 to 1.7e-3 off, at or below the output's own rounding
//     (1.7e-3).
//   * fp32 and fp16 output, and matrices of up to kSmallRows rows, whose time
//     goes to latency and not to products: hi lo + lo hi + hi hi, 22 bits.
//     The tensor cores' fp32 accumulation cuts off instead of rounding, half a
//     unit of the sum lost per MMA on average (2.2e-5 off the result at K =
//     4099 x 3), so the hi hi products are accumulated in chunks of 64 values
//     of K or fewer, added up in registers with rounding: as exact as fp32
//     products of the same formula (0.4 to 1.2 times their error; with chunks
//     of 128 up to 2.4 times it for n >> m, where A's large diagonal makes the
//     losses of A^2 agree, at the same time but for 4096^2 fp32, 3.1 to 3.2 ms).  The cross products, 2^-11 of the sum, have an
//     accumulator of their own.
//
// Measured (five steps; the floor is 5 (4 m^2 n) operations at the bf16 rate of
// 1900 TFLOP/s with the triangles, three times that for split products):
// 4096^2 bf16 1.10 to 1.13 ms (0.72), 4096^2 fp32 3.2 ms (2.2), 2048^2 bf16
// 250 us (90), 1000 x 4099 fp32 311 us (105), 12 x 1030 x 515 bf16 241 us (30),
// 256^2 106 us: rounds of tiles that are not full at the large ends, and at the
// small ones 15 products in a row, of which each has 1.1 us of first loads, 0.5
// to 2.8 us of joining and 1.1 to 1.8 us from one launch's end to the next.
//
// Two product kernels share one epilogue, value = c_old * old + c_acc * sum,
// stored as hi (and lo), at its mirror place too for the symmetric products,
// or as the result: `pair` (256 x 256 tiles on CTA pairs, persistent) where
// there are enough tiles to fill the machine, `tile` (128 x 128 tiles, K shared
// by a cluster and joined through distributed shared memory in a fixed order)
// below; every launch is a programmatic dependent of the one before.  Up to 128
// rows one launch of a third kernel does all of it on chip.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "ptx.cuh"

namespace dga {

__device__ int g_ns_status;  // non-zero: a bounded wait expired (role code)

namespace {

constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s
constexpr float kScale = 4096.0f;                 // stored = kScale * value
constexpr int kSmallRows = 256;
constexpr uint32_t kChunk = 1;  // K blocks of one chunk of the hi hi product where operands are split
constexpr uint32_t kBoxBytes = 64 * 64 * 2;  // an MN-major box: 64 columns x 64 k
enum : int { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3 };

struct NsParams {
    // tiles: of each matrix, all tiles_m x tiles_n or, sym, those with tm <= tn
    uint32_t tiles_m, tiles_n, sym, per_matrix, num_tiles;
    uint32_t num_kb;        // K blocks of 64
    uint32_t split;         // hi hi + hi lo + lo hi, else hi hi alone
    uint32_t q_mn;          // the second operand is read MN-major (rows along K)
    uint32_t p_rows, q_rows;  // rows of one matrix in each operand's map
    int32_t rows, ld;         // padded rows and columns of the value
    // value = c_old * (old hi + lo) + c_acc * sum
    float c_old, c_acc;
    uint32_t has_old, old_lo;  // there is an old value; it has a lo word
    uint32_t out_lo;           // the value is stored with its lo word
    uint32_t last;             // the value is the result
    void* result;
    int result_type, transposed;
    uint32_t result_tma, result_vec;  // its rows can be stored by TMA; by 16-byte stores
    int64_t m, n, ldo, stride_o;
};

__device__ __forceinline__ void record_failure(int role, volatile int* abort_flag) {
    atomicCAS(&g_ns_status, 0, role);
    *abort_flag = 1;
}

// kPer: tiles' columns to one tile's rows
template <uint32_t kPer = 1>
__device__ __forceinline__ void ns_tile(const NsParams& p, uint32_t t, uint32_t& matrix, uint32_t& tm, uint32_t& tn) {
    matrix = t / p.per_matrix;
    const uint32_t r = t - matrix * p.per_matrix;
    if (p.sym) {
        // column by column of the upper triangle of squares: square column c
        // has c + 1 of them, and begins at kPer c (c + 1) / 2
        uint32_t c = static_cast<uint32_t>((sqrtf(8.0f / kPer * static_cast<float>(r) + 1.0f) - 1.0f) * 0.5f);
        while (kPer * c * (c + 1) / 2 > r) --c;
        while (kPer * (c + 1) * (c + 2) / 2 <= r) ++c;
        const uint32_t at = r - kPer * c * (c + 1) / 2;
        tn = kPer * c + at / (c + 1);
        tm = at % (c + 1);
    } else {
        tm = r % p.tiles_m;
        tn = r / p.tiles_m;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// n columns of a row of X to the result: rows of m x n, or (transposed) of n x m.
template <typename T, int n>
__device__ __forceinline__ void ns_result(const NsParams& p, uint32_t matrix, int64_t row, int64_t col, const float (&v)[n]) {
    T* base = static_cast<T*>(p.result) + matrix * p.stride_o;
    if (p.transposed) {
        // element (col + j, row): consecutive lanes on consecutive columns
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (col + j < p.n) OutT<T>::store(base + (col + j) * p.ldo + row, v[j]);
    } else if (p.result_vec && col + n <= p.n) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int q = 0; q < n / kPer; ++q) {
            T w[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) OutT<T>::store(&w[e], v[q * kPer + e]);
            uint4 x;
            memcpy(&x, w, 16);
            *reinterpret_cast<uint4*>(base + row * p.ldo + col + q * kPer) = x;
        }
    } else {
#pragma unroll
        for (int j = 0; j < n; ++j)
            if (col + j < p.n) OutT<T>::store(base + row * p.ldo + col + j, v[j]);
    }
}

// The tensor maps of one product.  Operands: boxes of one 128-byte row of K
// (64 fp16) x 128 rows, or, MN-major, 64 columns x 64 rows of K.  Values: 32 x
// 32 of one matrix, so that what lies past a matrix' padded rows is neither
// read nor written.
struct NsMaps {
    CUtensorMap p_h, p_l, q_h, q_l, q64_h, q64_l, old_h, old_l, out_h, out_l, mirror_h, mirror_l, result;
};

// Byte offset of 16-byte piece `piece` (8 fp16) of a row in a box of 128-byte rows.
__device__ __forceinline__ uint32_t box_at(int row, int piece) {
    return static_cast<uint32_t>(row) * 128u + (static_cast<uint32_t>(piece ^ (row & 7)) << 4);
}
// Eight values as hi and lo.
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        h[j] = pack2(v[2 * j], v[2 * j + 1]);
        const float2 f = unpack2(h[j]);
        l[j] = pack2(v[2 * j] - f.x, v[2 * j + 1] - f.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// x[0..7] <- c_old * (hi + lo) + c_acc * x
__device__ __forceinline__ void blend8(float* x, const uint4& hi, const uint4& lo, float c_old, float c_acc) {
    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 a = unpack2(h[j]), b = unpack2(l[j]);
        x[2 * j] = fmaf(c_old, a.x + b.x, c_acc * x[2 * j]);
        x[2 * j + 1] = fmaf(c_old, a.y + b.y, c_acc * x[2 * j + 1]);
    }
}

// ---- the epilogue: units of 32 rows x 32 columns, one warp each ----------------------------
//
// A warp has two boxes of 32 rows x 64 bytes.  The old values come into them
// by TMA while the products run (hi, lo); lane l then takes row l's, in
// swizzled 16-byte pieces, and puts the new ones there, which TMA stores.
// (With a lane's own 16-byte loads and stores, one row per lane, the epilogue
// was bound by the L1's one line per cycle: 8,000 to 20,000 clocks a tile.)
constexpr uint32_t kBox32 = 32 * 64;
constexpr uint32_t kUnitBytes = 2 * kBox32;

// Byte offset of 16-byte piece `piece` (8 fp16) of a row in a box of 64-byte rows.
__device__ __forceinline__ uint32_t unit_at(int row, int piece) {
    return static_cast<uint32_t>(row) * 64u + (static_cast<uint32_t>(piece ^ ((row >> 1) & 3)) << 4);
}

// Starts the loads of a unit's old values (one lane).
__device__ __forceinline__ void unit_prefetch(const NsParams& p, const NsMaps& maps, uint8_t* boxes, uint64_t* bar,
                                              uint32_t matrix, int32_t row0, int32_t col0) {
    mbar_arrive_expect_tx(bar, p.old_lo ? 2 * kBox32 : kBox32);
    tma_load_3d(boxes, &maps.old_h, bar, col0, row0, static_cast<int32_t>(matrix));
    if (p.old_lo) tma_load_3d(boxes + kBox32, &maps.old_l, bar, col0, row0, static_cast<int32_t>(matrix));
}

// The result's part of ns_unit: v to rows of m x n, or (transposed) of n x m.
template <typename T>
__device__ __forceinline__ void unit_result(const NsParams& p, const NsMaps& maps, uint8_t* boxes, uint32_t matrix,
                                            int32_t row0, int32_t col0, int lane, const float (&v)[32]) {
    constexpr int kPer = 16 / sizeof(T);
    // fp32 rows are 128 bytes and take both boxes
    auto at = [](int row, int piece) { return sizeof(T) == 4 ? box_at(row, piece) : unit_at(row, piece); };
    if (p.transposed) {
        // column j of the unit becomes a row of 32
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const uint32_t to = smem_u32(boxes) + (j * 32 + lane) * sizeof(T);
            T x;
            OutT<T>::store(&x, v[j]);
            if constexpr (sizeof(T) == 4) {
                st_shared_u32(to, __float_as_uint(x));
            } else {
                uint16_t bits;
                memcpy(&bits, &x, 2);
                st_shared_u16(to, bits);
            }
        }
    } else {
#pragma unroll
        for (int q = 0; q < 32 / kPer; ++q) {
            T w[kPer];
#pragma unroll
            for (int e = 0; e < kPer; ++e) OutT<T>::store(&w[e], v[q * kPer + e]);
            uint4 x;
            memcpy(&x, w, 16);
            st_shared_v4(smem_u32(boxes) + at(lane, q), x);
        }
    }
    if (p.result_tma) {
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (row0 < p.m && col0 < p.n)
                tma_store_3d(&maps.result, boxes, p.transposed ? row0 : col0, p.transposed ? col0 : row0, static_cast<int32_t>(matrix));
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    T* base = static_cast<T*>(p.result) + matrix * p.stride_o;
    if (p.transposed) {
        if (row0 + lane < p.m)
            for (int j = 0; j < 32 && col0 + j < p.n; ++j)
                base[static_cast<int64_t>(col0 + j) * p.ldo + row0 + lane] = reinterpret_cast<const T*>(boxes)[j * 32 + lane];
    } else if (col0 + lane < p.n) {
        for (int i = 0; i < 32 && row0 + i < p.m; ++i)
            base[static_cast<int64_t>(row0 + i) * p.ldo + col0 + lane] =
                *reinterpret_cast<const T*>(boxes + at(i, lane / kPer) + (lane % kPer) * sizeof(T));
    }
    fence_async_shared();  // loads of old values may follow into these boxes
    __syncwarp();
}

// One unit of a tile, v its sums: lane l has row row0 + l, columns col0 ..
// col0 + 31.  mirror: the tile is off the diagonal of a symmetric product, so
// that its transpose is stored too.  free_groups: of this thread's bulk groups,
// the latest that do not use these boxes (2: none does).  `loaded` is called once the old values
// have been taken (by every lane).  On return the boxes' stores are under way,
// at most one bulk group of them (an earlier one has been waited for).
template <typename F>
__device__ __forceinline__ void ns_unit(const NsParams& p, const NsMaps& maps, uint8_t* boxes, uint64_t* bar, uint32_t phase,
                                        volatile int* abort_flag, uint32_t matrix, int32_t row0, int32_t col0, int lane,
                                        bool mirror, int free_groups, float (&v)[32], F loaded) {
    const uint32_t box = smem_u32(boxes);
    if (p.has_old) {
        if (!mbar_wait_bounded(bar, phase, abort_flag, kWaitLimitNs)) record_failure(kRoleEpilogue, abort_flag);
        uint4 lo = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 hi = ld_shared_v4(box + unit_at(lane, q));
            if (p.old_lo) lo = ld_shared_v4(box + kBox32 + unit_at(lane, q));
            blend8(&v[q * 8], hi, lo, p.c_old, p.c_acc);
        }
    } else {
        // the boxes may still be read by earlier stores
        if (lane == 0 && free_groups == 0) bulk_wait_read<0>();
        if (lane == 0 && free_groups == 1) bulk_wait_read<1>();
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] *= p.c_acc;
    }
    __syncwarp();
    loaded();
    if (p.last) {
        if (p.result_type == DGA_F32) unit_result<float>(p, maps, boxes, matrix, row0, col0, lane, v);
        else if (p.result_type == DGA_BF16) unit_result<__nv_bfloat16>(p, maps, boxes, matrix, row0, col0, lane, v);
        else unit_result<__half>(p, maps, boxes, matrix, row0, col0, lane, v);
        return;
    }
    uint32_t h[16], l[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint4 hi, lo;
        split8(&v[q * 8], hi, lo);
        st_shared_v4(box + unit_at(lane, q), hi);
        if (p.out_lo) st_shared_v4(box + kBox32 + unit_at(lane, q), lo);
        h[4 * q] = hi.x, h[4 * q + 1] = hi.y, h[4 * q + 2] = hi.z, h[4 * q + 3] = hi.w;
        l[4 * q] = lo.x, l[4 * q + 1] = lo.y, l[4 * q + 2] = lo.z, l[4 * q + 3] = lo.w;
    }
    fence_async_shared();
    __syncwarp();
    const bool in = row0 < p.rows && col0 < p.ld;
    if (lane == 0) {
        if (in) tma_store_3d(&maps.out_h, boxes, col0, row0, static_cast<int32_t>(matrix));
        if (in && p.out_lo) tma_store_3d(&maps.out_l, boxes + kBox32, col0, row0, static_cast<int32_t>(matrix));
        if (!mirror || p.out_lo) bulk_commit();
    }
    if (mirror) {
        // column j of the unit becomes a row of 32, hi in the second box if
        // there is no lo
        uint8_t* mh = p.out_lo ? boxes : boxes + kBox32;
        uint8_t* ml = boxes + kBox32;
        const uint32_t mh_s = smem_u32(mh) + lane * 2, ml_s = smem_u32(ml) + lane * 2;
        if (p.out_lo) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            st_shared_u16(mh_s + j * 64, j & 1 ? h[j / 2] >> 16 : h[j / 2]);
            if (p.out_lo) st_shared_u16(ml_s + j * 64, j & 1 ? l[j / 2] >> 16 : l[j / 2]);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (in) tma_store_3d(&maps.mirror_h, mh, row0, col0, static_cast<int32_t>(matrix));
            if (in && p.out_lo) tma_store_3d(&maps.mirror_l, ml, row0, col0, static_cast<int32_t>(matrix));
            bulk_commit();
        }
    }
}

// ---- the tile kernel: 128 x 128, K parts in a cluster ---------------------------------

// A ring slot holds the P and the Q box of a K block; split operands take two
// slots for it, the hi boxes and the lo boxes (each loaded once for the three
// products).  A CTA takes in 46 to 60 bytes a clock, which bounds these tiles:
// 512 clocks or more for a slot, whose MMAs take 256.
// kN: the tile's columns, 128 or, where K is short, 64: more tiles instead of
// parts of K, whose joining costs more than what is loaded twice then (2.8 us of a
// product's 7).
template <uint32_t kN>
struct TileShape {
    static constexpr int kStages = kN == 128 ? 5 : 8;
    static constexpr uint32_t kQ = kN * 128, kStage = 128 * 128 + kQ;
    static constexpr int kUnits = 4 * kN / 32;  // of 32 x 32, one to an epilogue warp
    static constexpr int kThreads = 64 + 32 * kUnits;  // and a producer and an MMA warp
    static constexpr uint32_t kEpi = kStages * kStage;
    static constexpr uint32_t kBar = kEpi + kUnits * kUnitBytes;
    // full[S], empty[S], acc_full[2], acc_empty[2], joined, old_full[U], then tmem slot + abort flag
    static constexpr uint32_t kLaunch = kBar + (2 * kStages + 5 + kUnits) * 8 + 16 + 1024;
};
constexpr uint32_t kUnitSums = 32 * 32 * 4;  // a unit's sums
static_assert(TileShape<128>::kEpi >= 2 * TileShape<128>::kUnits * kUnitSums, "the parts' sums fit the ring twice");

template <bool kSplit, uint32_t kN>
__global__ void __launch_bounds__(TileShape<kN>::kThreads, 1)
    ns_tile_kernel(const __grid_constant__ NsMaps maps, NsParams p, uint32_t k_parts) {
    const uint32_t splits = kN == 128 ? k_parts : 1;
    using S = TileShape<kN>;
    constexpr int kTileStages = S::kStages, kTileUnits = S::kUnits;
    constexpr uint32_t kTileStage = S::kStage, kTileEpi = S::kEpi;
    constexpr uint32_t kIdesc = idesc_mma(kFmtF16, 128, kN);
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBar);
    uint64_t* empty = full + kTileStages;
    uint64_t* acc_full = empty + kTileStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* joined = acc_empty + 2;
    uint64_t* old_full = joined + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(old_full + kTileUnits);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    // accumulators: one, or the cross products' and two for the chunks in turn
    constexpr uint32_t kCols = kSplit ? 4 * kN : kN;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x / splits, part = blockIdx.x % splits;
    const uint32_t kb0 = part * p.num_kb / splits, kb1 = (part + 1) * p.num_kb / splits;
    const uint32_t units = kTileUnits / splits;  // of the tile's, what this CTA joins and stores
    uint32_t matrix, tm, tn;
    ns_tile<128 / kN>(p, t, matrix, tm, tn);

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kTileStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], kTileUnits);
        }
        for (int w = 0; w < kTileUnits; ++w) mbar_init(&old_full[w], 1);
        mbar_init(joined, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if (splits > 1) mbar_arrive_expect_tx(joined, (splits - 1) * units * kUnitSums);
        tma_prefetch_desc(&maps.p_h);
        tma_prefetch_desc(&maps.q_h);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            const int32_t p_row = static_cast<int32_t>(matrix * p.p_rows + tm * 128);
            const uint32_t per = kSplit ? 2 : 1;  // slots of a K block
            for (uint32_t i = kb0 * per; i < kb1 * per; ++i) {
                if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleProducer, abort_flag);
                    __nanosleep(20000);  // let copies already issued land
                    break;
                }
                uint8_t* dst = smem + stage * kTileStage;
                mbar_arrive_expect_tx(&full[stage], kTileStage);
                const bool lo = kSplit && (i & 1);
                const int32_t k = static_cast<int32_t>((kSplit ? i >> 1 : i) * 64);
                tma_load_2d(dst, lo ? &maps.p_l : &maps.p_h, &full[stage], k, p_row);
                const CUtensorMap* q = lo ? &maps.q_l : &maps.q_h;
                if constexpr (kN == 64) {  // one box of 64 x 64 either way
                    const int32_t row = static_cast<int32_t>(matrix * p.q_rows);
                    const int32_t col = static_cast<int32_t>(tn * 64);
                    tma_load_2d(dst + 128 * 128, lo ? &maps.q64_l : &maps.q64_h, &full[stage], p.q_mn ? col : k, p.q_mn ? row + k : row + col);
                } else if (p.q_mn) {
                    const int32_t row = static_cast<int32_t>(matrix * p.q_rows) + k;
                    tma_load_2d(dst + 128 * 128, q, &full[stage], static_cast<int32_t>(tn * 128), row);
                    tma_load_2d(dst + 128 * 128 + kBoxBytes, q, &full[stage], static_cast<int32_t>(tn * 128 + 64), row);
                } else {
                    tma_load_2d(dst + 128 * 128, q, &full[stage], k, static_cast<int32_t>(matrix * p.q_rows + tn * 128));
                }
                if (++stage == kTileStages) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, chunk = 0;
            const uint32_t idesc = idesc_major(kIdesc, 0, p.q_mn);
            const uint32_t q_step = p.q_mn ? (16 * 128) >> 4 : 32 >> 4;
            auto mma = [&](uint32_t acc, uint32_t ps, uint32_t qs, bool fresh) {
                const uint32_t pa = smem_u32(smem + ps * kTileStage), qa = smem_u32(smem + qs * kTileStage) + 128 * 128;
                const uint64_t pd = smem_desc_kmajor_sw128(pa);
                const uint64_t qd = p.q_mn ? smem_desc_mnmajor_sw128(qa, kBoxBytes) : smem_desc_kmajor_sw128(qa);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma<kFmtF16>(tmem + acc, pd + 2 * k, qd + q_step * k, idesc, (fresh && k == 0) ? 0u : 1u);
            };
            auto next_full = [&](uint32_t& slot) {
                slot = stage;
                const bool ok = mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs);
                if (++stage == kTileStages) { stage = 0; phase ^= 1; }
                return ok;
            };
            for (uint32_t kb = kb0; kb < kb1; ++kb) {
                uint32_t hi = 0, lo = 0;
                if constexpr (kSplit) {
                    const bool begins = (kb - kb0) % kChunk == 0;
                    if (!next_full(hi) || !next_full(lo) ||
                        (begins && !mbar_wait_bounded(&acc_empty[chunk & 1], (chunk >> 1 & 1) ^ 1, abort_flag, kWaitLimitNs))) {
                        record_failure(kRoleMma, abort_flag);
                        __nanosleep(200000);  // let the MMAs issued finish
                        break;
                    }
                    tc_fence_after();
                    mma(0, hi, lo, kb == kb0);
                    mma(0, lo, hi, false);
                    mma(kN + (chunk & 1) * kN, hi, hi, begins);
                    tc_commit(&empty[hi]);
                    tc_commit(&empty[lo]);
                    if ((kb - kb0) % kChunk == kChunk - 1 || kb + 1 == kb1) {
                        tc_commit(&acc_full[chunk & 1]);
                        ++chunk;
                    }
                } else {
                    if (!next_full(hi)) {
                        record_failure(kRoleMma, abort_flag);
                        break;
                    }
                    tc_fence_after();
                    mma(0, hi, hi, kb == kb0);
                    tc_commit(&empty[hi]);
                }
            }
            if (!kSplit) tc_commit(&acc_full[0]);
        }
    }
    __syncwarp();
    if (warp >= 2) {
        // Unit (quarter, block): 32 rows, 32 columns.  With K in parts, CTA c
        // joins the blocks q % splits == c, whose warps keep their own sums;
        // once every CTA's ring is done with, the other warps send theirs by
        // bulk copies from the ring's first half to the second halves of the
        // joining CTAs, which add them up in the parts' order.
        const uint32_t e = warp - 2, quarter = warp & 3, block = e >> 2;
        const uint32_t lane_base = (quarter * 32) << 16;
        const bool joins = block % splits == part;
        const uint32_t slot = block / splits * 4 + quarter;  // at the joining CTA
        const int32_t row0 = static_cast<int32_t>(tm * 128 + quarter * 32), col0 = static_cast<int32_t>(tn * kN + block * 32);
        uint8_t* boxes = smem + kTileEpi + e * kUnitBytes;
        if (p.has_old && joins && lane == 0) unit_prefetch(p, maps, boxes, &old_full[e], matrix, row0, col0);
        __syncwarp();
        float v[32];
        auto add = [&](uint32_t column) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + lane_base + column + block * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += __uint_as_float(r[j]);
        };
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        const uint32_t n_chunks = kSplit ? (kb1 - kb0 + kChunk - 1) / kChunk : 1;
        for (uint32_t ch = 0; ch < n_chunks; ++ch) {
            if (!mbar_wait_bounded(&acc_full[ch & 1], ch >> 1 & 1, abort_flag, kWaitLimitNs)) {
                record_failure(kRoleEpilogue, abort_flag);
                break;
            }
            tc_fence_after();
            if constexpr (kSplit) {
                add(kN + (ch & 1) * kN);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[ch & 1]);
            }
        }
        add(0);
        if (splits > 1) {
            uint8_t* sent = smem + e * kUnitSums;
            if (!joins) {
#pragma unroll
                for (int j = 0; j < 32; ++j) st_shared_u32(smem_u32(sent) + (j * 32 + lane) * 4, __float_as_uint(v[j]));
                fence_async_shared();
            }
            __syncwarp();
            cluster_arrive();
            cluster_wait();  // every ring is done with
            if (!joins && lane == 0) {
                const uint32_t to = block % splits, at = smem_u32(smem + (kTileUnits + part * units + slot) * kUnitSums);
                bulk_copy_to_cta(map_to_cta(at, to), smem_u32(sent), kUnitSums, map_to_cta(smem_u32(joined), to));
            }
            __syncwarp();
            if (joins) {
                if (!mbar_wait_bounded<true>(joined, 0, abort_flag, kWaitLimitNs)) record_failure(kRoleEpilogue, abort_flag);
                float sum[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) sum[j] = 0.0f;
                for (uint32_t q = 0; q < splits; ++q) {
                    const uint32_t src = smem_u32(smem + (kTileUnits + q * units + slot) * kUnitSums) + lane * 4;
#pragma unroll
                    for (int j = 0; j < 32; ++j) sum[j] += q == part ? v[j] : ld_shared_f32(src + j * 128);
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = sum[j];
            }
            __syncwarp();
            cluster_arrive_relaxed();  // what was sent here has arrived
        }
        if (joins) {
            ns_unit(p, maps, boxes, &old_full[e], 0, abort_flag, matrix, row0, col0, lane, p.sym && tm != tn / (128 / kN), 2, v, [] {});
            if (lane == 0) bulk_wait_read<0>();  // shared memory outlives the stores that read it
        }
        __syncwarp();
        if (splits > 1) cluster_wait();  // and what this CTA sent, at the others
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
        tmem_dealloc(tmem, kCols);
    }
}

// ---- the pair kernel: 256 x 256 on two CTAs, persistent --------------------------------

// Warps: producer, MMA, 16 epilogue warps of 64 columns (two units) each, or,
// where each keeps its sums in registers, 8 of 128 (four units).  A unit's time
// is latency more than instructions, so warps count: with
// 8 warps for all, 12 x 1030 x 515 took 277 us instead of 240 to 260.
// Their 16 pairs of boxes make one for a warp, or two, so that one unit's old
// values arrive while another is computed; in a CTA's last tile, whose epilogue
// nothing hides, the remaining units take the ring's space, done with by then.
constexpr uint32_t kPairStage = 2 * 128 * 128;  // each CTA's half of both operands
constexpr int kPairStages = 5;
constexpr uint32_t kPairBoxes = 16;  // pairs of boxes
template <bool kSplit>
constexpr uint32_t kPairWarps = kSplit ? 8 : 16;
template <bool kSplit>
constexpr int kPairThreads = 64 + 32 * kPairWarps<kSplit>;
constexpr uint32_t kPairEpi = kPairStages * kPairStage;
constexpr uint32_t kPairBar = kPairEpi + kPairBoxes * kUnitBytes;
constexpr uint32_t kPairAllUnits = 32;  // of a CTA's 128 x 256
static_assert(kPairEpi >= kPairBoxes * kUnitBytes, "the last tile's boxes fit the ring");
// full[S], empty[S], acc_full[2], acc_empty[2], drain, old_full[units], tmem slot + abort flag
constexpr uint32_t kPairLaunch = kPairBar + (2 * kPairStages + 5 + kPairAllUnits) * 8 + 16 + 1024;

template <bool kSplit>
__global__ void __launch_bounds__(kPairThreads<kSplit>, 1)
    ns_pair_kernel(const __grid_constant__ NsMaps maps, NsParams p) {
    constexpr uint32_t kIdesc = idesc_mma(kFmtF16, 256, 256);
    constexpr uint16_t kBothCtas = 0x3;
    constexpr uint32_t kWarps = kPairWarps<kSplit>, kUnits = kPairAllUnits / kWarps, kSets = kPairBoxes / kWarps;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kPairBar);
    uint64_t* empty = full + kPairStages;
    uint64_t* acc_full = empty + kPairStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint64_t* old_full = drain + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(old_full + kPairAllUnits);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kPairStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kWarps);  // one lane of each epilogue warp of both CTAs
        }
        mbar_init(drain, 1);
        for (uint32_t w = 0; w < kPairAllUnits; ++w) mbar_init(&old_full[w], 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.p_h);
        tma_prefetch_desc(&maps.q_h);
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t cluster_id = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
    // accumulators of 256 columns: two in turn, or the cross products' and the chunks'

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            bool ok = true;
            for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters) {
                uint32_t matrix, tm, tn;
                ns_tile(p, t, matrix, tm, tn);
                const int32_t p_row = static_cast<int32_t>(matrix * p.p_rows + tm * 256 + rank * 128);
                const int32_t q_at = static_cast<int32_t>(tn * 256 + rank * 128);
                const int32_t q_row = static_cast<int32_t>(matrix * p.q_rows);
                const uint32_t per = kSplit ? 2 : 1;  // slots of a K block: the hi boxes, the lo boxes
                for (uint32_t i = 0; i < p.num_kb * per; ++i) {
                    if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleProducer, abort_flag);
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + stage * kPairStage;
                    if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kPairStage);
                    const uint32_t bar = map_to_cta(smem_u32(&full[stage]), 0);
                    const bool lo = kSplit && (i & 1);
                    const int32_t k = static_cast<int32_t>((kSplit ? i >> 1 : i) * 64);
                    tma_load_2d_pair(dst, lo ? &maps.p_l : &maps.p_h, bar, k, p_row);
                    const CUtensorMap* q = lo ? &maps.q_l : &maps.q_h;
                    if (p.q_mn) {
                        tma_load_2d_pair(dst + 128 * 128, q, bar, q_at, q_row + k);
                        tma_load_2d_pair(dst + 128 * 128 + kBoxBytes, q, bar, q_at + 64, q_row + k);
                    } else {
                        tma_load_2d_pair(dst + 128 * 128, q, bar, k, q_row + q_at);
                    }
                    if (++stage == kPairStages) { stage = 0; phase ^= 1; }
                }
            }
            if (!ok) __nanosleep(20000);  // let copies already issued land before teardown
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            const uint32_t idesc = idesc_major(kIdesc, 0, p.q_mn);
            const uint32_t q_step = p.q_mn ? (16 * 128) >> 4 : 32 >> 4;
            auto mma = [&](uint32_t d, uint32_t ps, uint32_t qs, bool fresh) {
                const uint32_t pa = smem_u32(smem + ps * kPairStage), qa = smem_u32(smem + qs * kPairStage) + 128 * 128;
                const uint64_t pd = smem_desc_kmajor_sw128(pa);
                const uint64_t qd = p.q_mn ? smem_desc_mnmajor_sw128(qa, kBoxBytes) : smem_desc_kmajor_sw128(qa);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_pair<kFmtF16>(tmem + d, pd + 2 * k, qd + q_step * k, idesc, (fresh && k == 0) ? 0u : 1u);
            };
            auto next_full = [&](uint32_t& slot) {
                slot = stage;
                const bool done = mbar_wait_bounded<true>(&full[stage], phase, abort_flag, kWaitLimitNs);
                if (++stage == kPairStages) { stage = 0; phase ^= 1; }
                return done;
            };
            auto acc_ready = [&]() { return mbar_wait_bounded<true>(&acc_empty[acc], acc_phase ^ 1, abort_flag, kWaitLimitNs); };
            bool ok = true;
            for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters) {
                for (uint32_t kb = 0; ok && kb < p.num_kb; ++kb) {
                    uint32_t hi = 0, lo = 0;
                    if constexpr (kSplit) {
                        // the chunks' accumulator is read while the next chunk's
                        // first cross products run; both are free at a tile's start
                        const bool begins = kb % kChunk == 0;
                        ok = next_full(hi) && next_full(lo) && (kb > 0 || acc_ready());
                        if (!ok) break;
                        tc_fence_after();
                        mma(0, hi, lo, kb == 0);
                        mma(0, lo, hi, false);
                        if (begins && kb > 0) {
                            ok = acc_ready();
                            if (!ok) break;
                            tc_fence_after();
                        }
                        mma(256, hi, hi, begins);
                        tc_commit_pair_multicast(&empty[hi], kBothCtas);
                        tc_commit_pair_multicast(&empty[lo], kBothCtas);
                        if (kb % kChunk == kChunk - 1 || kb + 1 == p.num_kb) {
                            tc_commit_pair_multicast(&acc_full[0], kBothCtas);
                            acc_phase ^= 1;
                        }
                    } else {
                        ok = (kb > 0 || acc_ready()) && next_full(hi);
                        if (!ok) break;
                        tc_fence_after();
                        mma(acc * 256, hi, hi, kb == 0);
                        tc_commit_pair_multicast(&empty[hi], kBothCtas);
                        if (kb + 1 == p.num_kb) {
                            tc_commit_pair_multicast(&acc_full[acc], kBothCtas);
                            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                        }
                    }
                }
            }
            if (!ok) record_failure(kRoleMma, abort_flag);
            tc_commit_pair_multicast(drain, 0x1);
            volatile int never = 0;
            mbar_wait_bounded(drain, 0, &never, kWaitLimitNs);
        }
    } else {
        const uint32_t e = warp - 2, quarter = warp & 3, share = e >> 2;  // kUnits * 32 columns
        const uint32_t lane_base = (quarter * 32) << 16;
        uint32_t acc = 0, acc_phase = 0, old_phase = 0;
        bool ok = true;
        auto boxes_of = [&](uint32_t u, bool last_tile) {
            return smem + (last_tile && u >= kSets ? 0 : kPairEpi) + (e * kSets + u % kSets) * kUnitBytes;
        };
        // unit u of tile t
        auto rows_of = [&](uint32_t tm) { return static_cast<int32_t>(tm * 256 + rank * 128 + quarter * 32); };
        auto cols_of = [&](uint32_t tn, uint32_t u) { return static_cast<int32_t>(tn * 256 + share * kUnits * 32 + u * 32); };
        auto in_range = [&](uint32_t tm, uint32_t tn, uint32_t u) {
            return rows_of(tm) < p.rows && cols_of(tn, u) < p.ld;
        };
        // the old values of unit u, once the boxes' last stores have been read
        auto prefetch = [&](uint32_t matrix, uint32_t tm, uint32_t tn, bool last_tile, uint32_t u) {
            if (p.has_old && lane == 0 && in_range(tm, tn, u)) {
                bulk_wait_read<0>();
                unit_prefetch(p, maps, boxes_of(u, last_tile), &old_full[e * kUnits + u], matrix, rows_of(tm), cols_of(tn, u));
            }
            __syncwarp();
        };
        auto prefetch_tile = [&](uint32_t t, uint32_t u) {
            if (p.has_old && t < p.num_tiles) {
                uint32_t matrix, tm, tn;
                ns_tile(p, t, matrix, tm, tn);
                prefetch(matrix, tm, tn, t + n_clusters >= p.num_tiles, u);
            }
        };
        for (uint32_t u = 0; u < kSets; ++u) prefetch_tile(cluster_id, u);
        for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters) {
            uint32_t matrix, tm, tn;
            ns_tile(p, t, matrix, tm, tn);
            const bool mirror = p.sym && tm != tn, last_tile = t + n_clusters >= p.num_tiles;
            float sum[kSplit ? kUnits : 1][32];
            if constexpr (kSplit) {
                auto add = [&](uint32_t column) {
#pragma unroll
                    for (uint32_t c = 0; c < kUnits; ++c) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(tmem + lane_base + column + share * kUnits * 32 + c * 32, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[c][j] += __uint_as_float(r[j]);
                    }
                };
#pragma unroll
                for (uint32_t j = 0; j < kUnits * 32; ++j) sum[j / 32][j % 32] = 0.0f;
                const uint32_t n_chunks = (p.num_kb + kChunk - 1) / kChunk;
                for (uint32_t ch = 0; ch < n_chunks; ++ch) {
                    if (!mbar_wait_bounded<true>(&acc_full[0], acc_phase, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleEpilogue, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    add(256);
                    if (ch + 1 == n_chunks) add(0);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_signal_cluster(map_to_cta(smem_u32(&acc_empty[0]), 0));
                    acc_phase ^= 1;
                }
            } else {
                if (!mbar_wait_bounded<true>(&acc_full[acc], acc_phase, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleEpilogue, abort_flag);
                    ok = false;
                }
                tc_fence_after();
            }
            if (!ok) break;
            if (last_tile)
                for (uint32_t u = kSets; u < kUnits; ++u) prefetch(matrix, tm, tn, true, u);
            // (one copy of the unit's code: unrolled, each would run once in a
            // launch and wait for its instructions)
#pragma unroll 1
            for (uint32_t u = 0; u < kUnits; ++u) {
                float v[32];
                if constexpr (kSplit) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        v[j] = sum[0][j];
#pragma unroll
                        for (uint32_t c = 1; c < kUnits; ++c) sum[c - 1][j] = sum[c][j];
                    }
                } else {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tmem + lane_base + acc * 256 + share * kUnits * 32 + u * 32, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    if (u == kUnits - 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_signal_cluster(map_to_cta(smem_u32(&acc_empty[acc]), 0));
                        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
                    }
                }
                // the next unit to load: into this one's boxes after it, or, of
                // two sets, into the other while this one is computed
                auto next = [&] {
                    if (last_tile) return;
                    if (u + 1 < kUnits) {
                        if (kSets == 1 || u > 0) prefetch(matrix, tm, tn, false, u + 1);
                    } else {
                        prefetch_tile(t + n_clusters, 0);
                    }
                };
                // a unit all of whose values lie past the matrix has nothing to do
                if (in_range(tm, tn, u)) {
                    ns_unit(p, maps, boxes_of(u, last_tile), &old_full[e * kUnits + u], old_phase >> u & 1, abort_flag, matrix,
                            rows_of(tm), cols_of(tn, u), lane, mirror, last_tile && u >= kSets ? 2 : static_cast<int>(kSets) - 1, v,
                            [&] { if (kSets > 1) next(); });
                    old_phase ^= 1u << u;
                    if (kSets == 1) next();
                } else {
                    next();
                }
            }
            if (kSets > 1) prefetch_tile(t + n_clusters, 1);
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

// ---- the norm and the first X ------------------------------------------------------------

template <typename T> __device__ __forceinline__ float ns_in(T v);
template <> __device__ __forceinline__ float ns_in<float>(float v) { return v; }
template <> __device__ __forceinline__ float ns_in<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float ns_in<__half>(__half v) { return __half2float(v); }

// The block's sum in every thread, in a fixed order.
template <int kWarps>
__device__ __forceinline__ float block_sum(float s) {
    __shared__ float part[kWarps];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w];
    return s;
}

// What G's values are multiplied by, from the sum of their squares: 0 where that
// passes fp32's range, which takes a norm of 0 and an eps next to it.
__device__ __forceinline__ float first_unit(float squares, float eps) {
    const float u = kScale / (sqrtf(squares) + eps);
    return u <= 3.4028235e38f || u != u ? u : 0.0f;
}

constexpr int64_t kSegment = 2048;  // columns of a row that a warp takes at once

// Eight consecutive values of a row from column c, zero from `cols` on.
template <typename T>
__device__ __forceinline__ void ns_load8(const T* row, int64_t c, int64_t cols, bool vec, float (&x)[8]) {
    if (vec && c + 8 <= cols) {
        T v[8];
        uint4 w[sizeof(T) / 2];
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T) / 2); ++q) w[q] = reinterpret_cast<const uint4*>(row + c)[q];
        memcpy(v, w, sizeof v);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = ns_in(v[q]);
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q) x[q] = c + q < cols ? ns_in(row[c + q]) : 0.0f;
    }
}

// Sums of squares of G (blockIdx.y: the matrix): each warp takes segments of
// rows in turn, a lane eight values at a time; one partial sum per block.
template <typename T>
__global__ void __launch_bounds__(256) ns_squares_kernel(const T* __restrict__ G, int64_t rows, int64_t cols,
                                                         int64_t ldg, int64_t stride_g, bool vec,
                                                         float* __restrict__ partial) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const T* base = G + blockIdx.y * stride_g;
    const int64_t segments = (cols + kSegment - 1) / kSegment, units = rows * segments;
    float s[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) s[q] = 0.0f;
    for (int64_t u = blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += gridDim.x * 8) {
        const int64_t r = u / segments, c0 = (u - r * segments) * kSegment;
        const int64_t end = min(cols, c0 + kSegment);
#pragma unroll 4
        for (int64_t c = c0 + (threadIdx.x & 31) * 8; c < end; c += 256) {
            float x[8];
            ns_load8(base + r * ldg, c, cols, vec, x);
#pragma unroll
            for (int q = 0; q < 8; ++q) s[q] = fmaf(x[q], x[q], s[q]);
        }
    }
    const float total = block_sum<8>(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
    if (threadIdx.x == 0) partial[blockIdx.y * gridDim.x + blockIdx.x] = total;
}

// X = G / (|G| + eps) as hi and lo, zero in the padding: 64 x 64 tiles, a
// thread 16 consecutive columns of a row; a tall G is transposed through
// shared memory.
template <typename T>
__global__ void __launch_bounds__(256) ns_first_kernel(const T* __restrict__ G, int64_t rows, int64_t cols, int64_t ldg,
                                                       int64_t stride_g, bool vec, bool transposed,
                                                       const float* __restrict__ partial, int parts, float eps,
                                                       __half* __restrict__ xh, __half* __restrict__ xl, int64_t ld,
                                                       int64_t stride, uint32_t tiles_c) {
    __shared__ float tile[64][65];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / tiles_c) * 64, c0 = static_cast<int64_t>(blockIdx.x % tiles_c) * 64;
    const int tr = threadIdx.x >> 2, tc = (threadIdx.x & 3) * 16;
    // X's rows r0.., columns c0..: G's rows from r0 (c0), columns from c0 (r0)
    const int64_t gr = (transposed ? c0 : r0) + tr, gc = (transposed ? r0 : c0) + tc;
    const T* row = G + blockIdx.y * stride_g + gr * ldg;
    float x[2][8];
#pragma unroll
    for (int q = 0; q < 2; ++q) ns_load8(row, gr < rows ? gc + q * 8 : cols, cols, vec, x[q]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.0f;
    for (int i = threadIdx.x; i < parts; i += 256) s += partial[blockIdx.y * parts + i];
    const float u = first_unit(block_sum<8>(s), eps);
    if (transposed) {
#pragma unroll
        for (int j = 0; j < 16; ++j) tile[tc + j][tr] = x[j / 8][j % 8];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j / 8][j % 8] = tile[tr][tc + j];
    }
    const int64_t at = blockIdx.y * stride + (r0 + tr) * ld + c0 + tc;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = x[q][2 * j] * u, b = x[q][2 * j + 1] * u;
            h[j] = pack2(a, b);
            const float2 f = unpack2(h[j]);
            l[j] = pack2(a - f.x, b - f.y);
        }
        *reinterpret_cast<uint4*>(xh + at + q * 8) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(xl + at + q * 8) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// ---- the cluster kernel: up to 128 rows, all steps in one launch -------------------------
//
// One cluster of C CTAs per matrix; each CTA keeps a slab of X's columns (up
// to 192) in its shared memory for all steps, as boxes of 64 columns x 128
// rows (128-byte swizzle rows), which the MMA reads K-major for X X^T and
// MN-major for B X.  A step is
//   1. each CTA's share of X X^T (its columns are a part of K);
//   2. the shares added up: CTA c receives columns [c 128/C, (c+1) 128/C) of
//      all of them (stores into its `red`), adds them in the CTAs' order, and
//      has A's rows of the same numbers (A is symmetric), as hi and lo: rows
//      of the boxes lie together, so that bulk copies hand them to the others;
//   3. A^2, B = b A + c A^2 and X <- a X + B X of the slab, in each CTA.
// Only step 2 crosses CTAs, with one full cluster barrier.  With C = 1 nothing
// does.  Accumulators: the cross products in one, the hi hi product
// in up to three, of 32 to 64 values of K each (B X: of 128).
// For m, n this small the time is latency: 15 products of 1 to 2 us and, with
// C > 1, an exchange of about 5 us a step.  29 us at 64 x 64, 59 us at 128 x
// 512; as separate launches (2 + 3 a step) 85 and 134 us.

constexpr int kMaxBoxes = 3;                      // 64-column boxes of a slab
constexpr int kMaxCluster = 16;
constexpr uint32_t kXBox = 128 * 128;             // bytes of a box: 128 rows x 64 fp16
constexpr uint32_t kABytes = 2 * kXBox;           // A or B, hi or lo
constexpr int kClusterThreads = 512;
static_assert(2 * kABytes == 128 * 128 * 4, "`red` has B's memory");

struct NsClusterParams {
    const void* G;
    int64_t ldg, stride_g;
    int64_t m, n;
    bool transposed, vec;
    int boxes_all, boxes_each, cluster;  // boxes of X, of a CTA's slab; CTAs
    float eps;
    int steps;
    float coefficients[3 * 32];
};

template <typename T>
__global__ void __launch_bounds__(kClusterThreads, 1) ns_cluster_kernel(NsClusterParams c, NsParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t done, gathered;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word;
    __shared__ float norms[kMaxCluster];
    volatile int* abort_flag = &abort_word;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int matrix = blockIdx.x / c.cluster, rank = blockIdx.x % c.cluster;
    const int first_box = rank * c.boxes_each;
    const int boxes = max(0, min(c.boxes_each, c.boxes_all - first_box));
    uint8_t* xh = smem;
    uint8_t* xl = xh + c.boxes_each * kXBox;
    uint8_t* ah = xl + c.boxes_each * kXBox;
    uint8_t* al = ah + kABytes;
    uint8_t* bh = al + kABytes;
    uint8_t* bl = bh + kABytes;

    if (tid == 0) {
        mbar_init(&done, 1);
        mbar_init(&gathered, 1);
        abort_word = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }

    // ---- X = G / (|G| + eps): the slab in registers, its norm, then hi and lo
    const T* G = static_cast<const T*>(c.G) + matrix * c.stride_g;
    const int64_t col0 = static_cast<int64_t>(first_box) * 64;
    float x[kMaxBoxes][2][8];
    float s = 0.0f;
    // not transposed: four threads to a row, 16 columns each; transposed: eight
    // to a column, 16 rows each
    const int line = c.transposed ? tid >> 3 : tid >> 2, at16 = c.transposed ? (tid & 7) * 16 : (tid & 3) * 16;
#pragma unroll
    for (int b = 0; b < kMaxBoxes; ++b) {
        if (b < boxes) {
            const int64_t gr = c.transposed ? col0 + b * 64 + line : line;
            const int64_t gc = c.transposed ? at16 : col0 + b * 64 + at16;
            const int64_t rows = c.transposed ? c.n : c.m, cols = c.transposed ? c.m : c.n;
#pragma unroll
            for (int q = 0; q < 2; ++q) ns_load8(G + gr * c.ldg, gr < rows ? gc + q * 8 : cols, cols, c.vec, x[b][q]);
        }
    }
#pragma unroll
    for (int b = 0; b < kMaxBoxes; ++b)
        if (b < boxes)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(x[b][q][j], x[b][q][j], s);
    s = block_sum<kClusterThreads / 32>(s);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (c.cluster > 1) {
        cluster_sync();  // every CTA of the cluster runs
        if (tid < c.cluster) st_shared_cluster_f32(map_to_cta(smem_u32(&norms[rank]), tid), s);
        cluster_sync();
        s = 0.0f;
        for (int q = 0; q < c.cluster; ++q) s += norms[q];
    }
    const float unit = first_unit(s, c.eps);
#pragma unroll
    for (int b = 0; b < kMaxBoxes; ++b) {
        if (b < boxes) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[b][q][j] *= unit;
                uint4 hi, lo;
                split8(x[b][q], hi, lo);
                if (!c.transposed) {
                    const uint32_t at = b * kXBox + box_at(line, (at16 >> 3) + q);
                    st_shared_v4(smem_u32(xh) + at, hi);
                    st_shared_v4(smem_u32(xl) + at, lo);
                } else {
                    const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t at = b * kXBox + box_at(at16 + q * 8 + j, line >> 3) + (line & 7) * 2;
                        st_shared_u16(smem_u32(xh) + at, j & 1 ? h[j / 2] >> 16 : h[j / 2]);
                        st_shared_u16(smem_u32(xl) + at, j & 1 ? l[j / 2] >> 16 : l[j / 2]);
                    }
                }
            }
        }
    }
    fence_async_shared();
    __syncthreads();

    const int quarter = warp & 3, group = warp >> 2;  // of 4 groups of warps
    const int row = quarter * 32 + lane;  // of A, B and X
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t xh_s = smem_u32(xh), xl_s = smem_u32(xl), ah_s = smem_u32(ah), al_s = smem_u32(al);
    const uint32_t bh_s = smem_u32(bh), bl_s = smem_u32(bl), red_s = bh_s;  // `red`: floats
    constexpr uint32_t kIdesc = idesc_mma(kFmtF16, 128, 128);
    uint32_t phase = 0;
    auto wait_done = [&]() {
        if (!mbar_wait_bounded(&done, phase, abort_flag, kWaitLimitNs)) record_failure(kRoleEpilogue, abort_flag);
        phase ^= 1;
        tc_fence_after();
    };
    // 16 columns of tensor memory from `a`, and from `b`, added up
    auto add16 = [&](uint32_t a, uint32_t b, float (&v)[16]) {
        uint32_t r[16], t[16];
        tmem_ld_32x32b_x16(tmem + lane_base + a, r);
        tmem_ld_32x32b_x16(tmem + lane_base + b, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]) + __uint_as_float(t[j]);
    };
    auto more16 = [&](uint32_t a, float (&v)[16]) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(tmem + lane_base + a, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
    };
    // D[128 x 128] (+)= P P'^T over `n` boxes of 64, both K-major
    auto mma_kk = [&](uint32_t acc, uint32_t pa, uint32_t qa, int n, bool fresh) {
        for (int b = 0; b < n; ++b) {
            const uint64_t pd = smem_desc_kmajor_sw128(pa + b * kXBox), qd = smem_desc_kmajor_sw128(qa + b * kXBox);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                tc_mma<kFmtF16>(tmem + acc, pd + 2 * k, qd + 2 * k, kIdesc, (fresh && b == 0 && k == 0) ? 0u : 1u);
        }
    };
    // The same for a symmetric hi hi product of n MMAs (16 of K each), in chunks
    // of `each` with an accumulator each: columns 128, 256 and 384 on.
    auto mma_chunks = [&](uint32_t pa, int n, int each) {
        uint32_t acc = tmem + 128;
        int left = each;
        for (int b = 0; b < n; b += 4) {
            const uint64_t d = smem_desc_kmajor_sw128(pa + (b >> 2) * kXBox);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (left == 0) {
                    acc += 128;
                    left = each;
                }
                tc_mma<kFmtF16>(acc, d + 2 * k, d + 2 * k, kIdesc, left == each ? 0u : 1u);
                --left;
            }
        }
    };
    // up to three chunks: of 64 of K, 48, 48 and 32, or 32
    const int x_each = boxes == 3 ? 4 : boxes == 2 ? 3 : 2, x_chunks = boxes > 1 ? 3 : 2;
    const int a_mmas = c.m <= 64 ? 4 : 8;  // of A^2: K to A's last box in use
    const int a_each = c.m <= 64 ? 2 : 3, a_chunks = c.m <= 64 ? 2 : 3;
    const int per = 128 / c.cluster, shift = 31 - __clz(per);  // columns of the shares, rows of A, that a CTA joins

    for (int step = 0; step < c.steps; ++step) {
        const float ca = c.coefficients[3 * step], cb = c.coefficients[3 * step + 1], cc = c.coefficients[3 * step + 2];
        // ---- 1. this CTA's share of X X^T: columns 0-127 the cross products, then 128 a chunk
        if (tid == 0 && boxes > 0) {
            mma_kk(0, xh_s, xl_s, boxes, true);
            mma_kk(0, xl_s, xh_s, boxes, false);
            mma_chunks(xh_s, 4 * boxes, x_each);
            tc_commit(&done);
        }
        __syncwarp();
        if (boxes > 0) wait_done();
        // ---- 2. the shares joined
        __syncwarp();
        if (c.cluster > 1 && step > 0) cluster_wait();  // every CTA is done with B, whose memory `red` is
#pragma unroll 1
        for (int b16 = group * 2; b16 < group * 2 + 2; ++b16) {
            float v[16];
            if (boxes > 0) {
                add16(b16 * 16, 128 + b16 * 16, v);
                for (int i = 1; i < x_chunks; ++i) more16(128 + 128 * i + b16 * 16, v);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = 0.0f;
            }
            if (c.cluster == 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] *= 1.0f / kScale;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint4 hi, lo;
                    split8(&v[q * 8], hi, lo);
                    const uint32_t at = (b16 >> 2) * kXBox + box_at(row, (b16 & 3) * 2 + q);
                    st_shared_v4(ah_s + at, hi);
                    st_shared_v4(al_s + at, lo);
                }
            } else {
                // red[(share * per + column) * 128 + row] of the joining CTA
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int col = b16 * 16 + q * 8;  // one CTA for 8 columns
                    const uint32_t to = map_to_cta(red_s + ((rank * per + (col & (per - 1))) * 128 + row) * 4, col >> shift);
#pragma unroll
                    for (int j = 0; j < 8; ++j) st_shared_cluster_f32(to + j * 512, v[q * 8 + j]);
                }
            }
        }
        if (c.cluster > 1) {
            __syncwarp();
            cluster_sync();
            if (tid == 0) mbar_arrive_expect_tx(&gathered, static_cast<uint32_t>((c.cluster - 1) * per * 512));
            // four columns of a row of A at a time
            for (int u = tid; u < per * 32; u += kClusterThreads) {
                const int r = u >> 5, col = (u & 31) * 4;
                float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                for (int share = 0; share < c.cluster; ++share) {
                    const uint4 x4 = ld_shared_v4(red_s + ((share * per + r) * 128 + col) * 4);
                    v[0] += __uint_as_float(x4.x);
                    v[1] += __uint_as_float(x4.y);
                    v[2] += __uint_as_float(x4.z);
                    v[3] += __uint_as_float(x4.w);
                }
                uint32_t h[2], l[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float a = v[2 * j] * (1.0f / kScale), b = v[2 * j + 1] * (1.0f / kScale);
                    h[j] = pack2(a, b);
                    const float2 f = unpack2(h[j]);
                    l[j] = pack2(a - f.x, b - f.y);
                }
                const uint32_t at = (col >> 6) * kXBox + box_at(rank * per + r, (col & 63) >> 3) + (col & 4) * 2;
                st_shared_v2(ah_s + at, h[0], h[1]);
                st_shared_v2(al_s + at, l[0], l[1]);
            }
            fence_async_shared();
            __syncthreads();
            // these rows, of both boxes of hi and lo (four runs of per * 128
            // bytes), to every other CTA
            if (tid < 4 * c.cluster && tid >> 2 != rank) {
                const uint32_t at = ah_s + (tid & 3) * kXBox + rank * per * 128;
                const uint32_t to = static_cast<uint32_t>(tid >> 2);
                bulk_copy_to_cta(map_to_cta(at, to), at, per * 128, map_to_cta(smem_u32(&gathered), to));
            }
            __syncwarp();
            if (!mbar_wait_bounded<true>(&gathered, step & 1, abort_flag, kWaitLimitNs)) record_failure(kRoleProducer, abort_flag);
        }
        tc_fence_before();
        fence_async_shared();
        __syncthreads();
        tc_fence_after();
        // ---- 3. B = b A + c A^2
        if (tid == 0) {
            mma_kk(0, ah_s, al_s, 2, true);
            mma_kk(0, al_s, ah_s, 2, false);
            mma_chunks(ah_s, a_mmas, a_each);
            tc_commit(&done);
        }
        __syncwarp();
        wait_done();
#pragma unroll 1
        for (int b16 = group * 2; b16 < group * 2 + 2; ++b16) {
            float v[16];
            add16(b16 * 16, 128 + b16 * 16, v);
            for (int i = 1; i < a_chunks; ++i) more16(128 + 128 * i + b16 * 16, v);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t at = (b16 >> 2) * kXBox + box_at(row, (b16 & 3) * 2 + q);
                uint4 hi = ld_shared_v4(ah_s + at), lo = ld_shared_v4(al_s + at);
                blend8(&v[q * 8], hi, lo, cb, cc / kScale);
                split8(&v[q * 8], hi, lo);
                st_shared_v4(bh_s + at, hi);
                st_shared_v4(bl_s + at, lo);
            }
        }
        tc_fence_before();
        fence_async_shared();
        __syncthreads();
        tc_fence_after();
        // ---- X <- a X + B X: cross products in columns 0-255, hi hi in 256-511
        if (boxes > 0) {
            if (tid == 0) {
                const uint32_t idesc = idesc_major(idesc_mma(kFmtF16, 128, static_cast<uint32_t>(boxes) * 64), 0, 1);
                auto mma_kn = [&](uint32_t acc, uint32_t pa, uint32_t qa, bool fresh) {
                    // K = 128 rows of X, 16 at a time: 32 bytes along B's rows, 16 rows of X's boxes
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint64_t pd = smem_desc_kmajor_sw128(pa + (k >> 2) * kXBox) + 2 * (k & 3);
                        const uint64_t qd = smem_desc_mnmajor_sw128(qa, kXBox) + 128 * k;
                        tc_mma<kFmtF16>(tmem + acc, pd, qd, idesc, (fresh && k == 0) ? 0u : 1u);
                    }
                };
                mma_kn(0, bh_s, xl_s, true);
                mma_kn(0, bl_s, xh_s, false);
                mma_kn(256, bh_s, xh_s, true);
                tc_commit(&done);
            }
            __syncwarp();
            wait_done();
        }
        const bool last = step + 1 == c.steps;
        __syncwarp();
        if (c.cluster > 1 && !last) cluster_arrive();  // this CTA is done with B
        if (boxes > 0) {
#pragma unroll 1
            for (int b16 = group * boxes; b16 < (group + 1) * boxes; ++b16) {
                float v[16];
                add16(b16 * 16, 256 + b16 * 16, v);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t at = (b16 >> 2) * kXBox + box_at(row, (b16 & 3) * 2 + q);
                    uint4 hi = ld_shared_v4(xh_s + at), lo = ld_shared_v4(xl_s + at);
                    if (last) {
                        blend8(&v[q * 8], hi, lo, ca / kScale, 1.0f / (kScale * kScale));
                    } else {
                        blend8(&v[q * 8], hi, lo, ca, 1.0f / kScale);
                        split8(&v[q * 8], hi, lo);
                        st_shared_v4(xh_s + at, hi);
                        st_shared_v4(xl_s + at, lo);
                    }
                }
                if (last && row < p.m) {
                    const int64_t col = col0 + b16 * 16;
                    if (p.result_type == DGA_F32) ns_result<float>(p, matrix, row, col, v);
                    else if (p.result_type == DGA_BF16) ns_result<__nv_bfloat16>(p, matrix, row, col, v);
                    else ns_result<__half>(p, matrix, row, col, v);
                }
            }
        }
        tc_fence_before();
        fence_async_shared();
        __syncthreads();
        tc_fence_after();
    }
    __syncwarp();
    if (c.cluster > 1) cluster_sync();  // no CTA leaves while another may still write to it
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem, 512);
    }
}

// ---- host side ------------------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// batch matrices of rows x cols values, boxes of 32 x 32 of one of them, whose
// rows in shared memory are swizzled or not.
cudaError_t value_map(CUtensorMap* map, int type, const void* base, int64_t cols, int64_t rows, int64_t batch, int64_t ld,
                      int64_t stride, bool swizzle) {
    auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t es = type == DGA_F32 ? 4 : 2;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(batch)};
    // a single matrix has no stride to speak of: any multiple of 16 bytes
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * es, batch > 1 ? static_cast<cuuint64_t>(stride) * es : static_cast<cuuint64_t>(ld) * es};
    cuuint32_t box[3] = {32, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(map, type == DGA_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : type == DGA_F32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// rows x ld fp16, boxes of 64 columns (one 128-byte row) x box_rows
cudaError_t half_map(CUtensorMap* map, const __half* base, int64_t rows, int64_t ld, uint32_t box_rows) {
    auto fn = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!fn) return cudaErrorNotSupported;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(ld), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    cuuint32_t box[2] = {64, box_rows};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

constexpr int kMaxParts = 512;  // partial sums of squares per matrix

struct NsPlan {
    int64_t m, n, mp, np;  // m <= n, and padded to the K block
    bool transposed, split;
    size_t x_bytes, a_bytes, total;  // one X (hi or lo), one A or B (hi or lo)
};

NsPlan plan_of(int out_dtype, int64_t batch, int64_t rows, int64_t cols) {
    NsPlan pl{};
    pl.transposed = rows > cols;
    pl.m = std::min(rows, cols);
    pl.n = std::max(rows, cols);
    pl.mp = round_up(pl.m, 64);
    pl.np = round_up(pl.n, 64);
    pl.split = out_dtype != DGA_BF16 || pl.m <= kSmallRows;
    pl.x_bytes = static_cast<size_t>(batch * pl.mp * pl.np) * 2;
    pl.a_bytes = static_cast<size_t>(batch * pl.mp * pl.mp) * 2;
    // partial sums; X now and next, hi and lo; A and B, hi and (split) lo
    pl.total = static_cast<size_t>(round_up(batch * kMaxParts * 4, 256)) + 4 * pl.x_bytes + (pl.split ? 4 : 2) * pl.a_bytes;
    return pl;
}

// most_smem: the most that any launch of this kernel takes.  The limit is set to
// that, not to this launch's share: another host thread's launch may come between.
template <typename... P, typename... A>
cudaError_t launch(void (*kern)(P...), dim3 grid, int threads, unsigned cluster, int smem, int most_smem, bool pdl, cudaStream_t s,
                   const A&... args) {
    if (smem > 0) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// One product: pair kernel where its tiles can occupy most of the machine's
// CTA pairs, else the tile kernel with K in parts.
cudaError_t launch_product(NsParams p, const NsMaps& maps, int64_t batch, int64_t rows, int64_t cols,
                           const DeviceInfo& dev, cudaStream_t s) {
    // tiles of 256 or 128 squared, or 128 x 64
    auto tiles = [&](int64_t size) {
        const int64_t high = std::max<int64_t>(size, 128);
        p.tiles_m = static_cast<uint32_t>((rows + high - 1) / high);
        p.tiles_n = static_cast<uint32_t>((cols + size - 1) / size);
        if (p.sym) {
            const uint32_t per = static_cast<uint32_t>(high / size), whole = p.tiles_n / per;  // columns of squares
            p.per_matrix = per * whole * (whole + 1) / 2 + p.tiles_n % per * (whole + 1);
        } else {
            p.per_matrix = p.tiles_m * p.tiles_n;
        }
        const int64_t all = batch * p.per_matrix;
        p.num_tiles = static_cast<uint32_t>(all);
        return all;
    };
    const int64_t pairs = dev.sm_count / 2;
    const int64_t big = tiles(256);
    if (big >= pairs * 3 / 4) {
        return launch(p.split ? ns_pair_kernel<true> : ns_pair_kernel<false>,
                      dim3(static_cast<unsigned>(2 * std::min(big, pairs))), p.split ? kPairThreads<true> : kPairThreads<false>, 2, static_cast<int>(kPairLaunch),
                      static_cast<int>(kPairLaunch), true, s, maps, p);
    }
    // Tiles of 64 columns where K is short and even they leave half of the SMs
    // idle (700^2 bf16 115 -> 101 us, 400 x 1000 bf16 109 -> 96 us, 150^2 fp32
    // 105 -> 92 us); split operands with more slots do better with parts of K
    // (256 x 512 fp32 111 us against 116 to 119).
    const uint32_t slots = p.num_kb * (p.split ? 2 : 1);
    if (slots <= (p.split ? 6u : 16u)) {
        const int64_t narrow = tiles(64);
        if (narrow * 2 <= dev.sm_count)
            return launch(p.split ? ns_tile_kernel<true, 64> : ns_tile_kernel<false, 64>, dim3(static_cast<unsigned>(narrow)),
                          TileShape<64>::kThreads, 1, static_cast<int>(TileShape<64>::kLaunch), static_cast<int>(TileShape<64>::kLaunch),
                          true, s, maps, p, 1u);
    }
    // Parts of K while there are idle SMs: joining them takes 2 to 3 us, a slot
    // 0.3 us.  Split operands with 8 slots or more gain from 4 parts (256^2 fp32
    // 133 -> 123 us, 400 x 1000 fp32 166 -> 147 us); single ones from 16 slots
    // to a part (700^2 bf16 119 us with, 132 us from 4 slots to a part).
    const int64_t small = tiles(128);
    uint32_t splits = 1;
    while (splits < 4 && small * splits * 2 <= dev.sm_count && slots >= (p.split ? 8u : splits * 16)) splits *= 2;
    return launch(p.split ? ns_tile_kernel<true, 128> : ns_tile_kernel<false, 128>, dim3(static_cast<unsigned>(small * splits)),
                  TileShape<128>::kThreads, splits, static_cast<int>(TileShape<128>::kLaunch), static_cast<int>(TileShape<128>::kLaunch),
                  true, s, maps, p, splits);
}

// The cluster kernel's shape, or cluster = 0 where it does not apply: up to 128
// rows and 16 slabs of 192 columns.  CTAs are added while a slab is over 128
// columns and the batch leaves room for them, and as far as the slabs need
// them; clusters of 16 only where the device can place one.
struct ClusterShape {
    int cluster, boxes_all, boxes_each, smem;
};
template <typename T>
bool places_16(int smem, const DeviceInfo& dev) {
    static int known[64] = {};  // 0 unknown, 1 no, 2 yes
    static std::mutex mu;
    std::lock_guard<std::mutex> lock(mu);
    int& k = known[dev.ordinal & 63];
    if (k == 0) {
        k = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kClusterThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(ns_cluster_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaFuncSetAttribute(ns_cluster_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, ns_cluster_kernel<T>, &cfg) == cudaSuccess && n > 0)
            k = 2;
        else
            cudaGetLastError();
    }
    return k == 2;
}
constexpr int cluster_smem(int boxes) { return static_cast<int>(2 * boxes * kXBox + 4 * kABytes + 1024); }
template <typename T>
ClusterShape cluster_shape(const OrthoArgs& a, const NsPlan& pl, const DeviceInfo& dev) {
    ClusterShape c{};
    if (pl.m > 128 || pl.np > kMaxCluster * 64 * kMaxBoxes || a.steps > 32) return c;
    c.boxes_all = static_cast<int>(pl.np / 64);
    auto each = [&](int n) { return (c.boxes_all + n - 1) / n; };
    int n = 1;
    while (n < 8 && each(n) > 2 && (each(n) > kMaxBoxes || a.batch * n * 2 <= dev.sm_count)) n *= 2;
    if (each(n) > kMaxBoxes) n = kMaxCluster;
    if (n == kMaxCluster && !places_16<T>(cluster_smem(kMaxBoxes), dev)) return c;
    c.cluster = n;
    c.boxes_each = each(n);
    c.smem = cluster_smem(c.boxes_each);
    return c;
}

template <typename T>
cudaError_t launch_cluster(const OrthoArgs& a, const NsPlan& pl, const NsParams& p, const DeviceInfo& dev, bool* done) {
    const ClusterShape shape = cluster_shape<T>(a, pl, dev);
    *done = shape.cluster > 0;
    if (!*done) return cudaSuccess;
    constexpr int64_t kVec = 16 / sizeof(T);
    NsClusterParams c{};
    c.G = a.G;
    c.ldg = a.ldg;
    c.stride_g = a.stride_g;
    c.m = pl.m;
    c.n = pl.n;
    c.transposed = pl.transposed;
    c.vec = aligned(a.G, 16) && a.ldg % kVec == 0 && (a.batch == 1 || a.stride_g % kVec == 0);
    c.boxes_all = shape.boxes_all;
    c.boxes_each = shape.boxes_each;
    c.cluster = shape.cluster;
    c.eps = a.eps;
    c.steps = a.steps;
    for (int i = 0; i < 3 * a.steps; ++i) c.coefficients[i] = a.coefficients[i];
    return launch(ns_cluster_kernel<T>, dim3(static_cast<unsigned>(a.batch * shape.cluster)), kClusterThreads, shape.cluster,
                  shape.smem, cluster_smem(kMaxBoxes), false, a.stream, c, p);
}

template <typename T>
cudaError_t launch_first(const OrthoArgs& a, const NsPlan& pl, float* partial, __half* xh, __half* xl,
                         const DeviceInfo& dev, cudaStream_t s) {
    const T* G = static_cast<const T*>(a.G);
    constexpr int64_t kVec = 16 / sizeof(T);
    const bool vec = aligned(G, 16) && a.ldg % kVec == 0 && (a.batch == 1 || a.stride_g % kVec == 0);
    // blocks of eight segments each, a few to an SM at most over all matrices
    const int64_t units = a.rows * ((a.cols + kSegment - 1) / kSegment);
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(kMaxParts, 4 * dev.sm_count / a.batch));
    const int parts = static_cast<int>(std::min<int64_t>((units + 7) / 8, most));
    cudaError_t e = launch(ns_squares_kernel<T>, dim3(parts, static_cast<unsigned>(a.batch)), 256, 1, 0, 0, false, s, G, a.rows,
                           a.cols, a.ldg, a.stride_g, vec, partial);
    if (e != cudaSuccess) return e;
    const uint32_t tiles_c = static_cast<uint32_t>(pl.np / 64);
    return launch(ns_first_kernel<T>, dim3(static_cast<unsigned>(pl.mp / 64 * tiles_c), static_cast<unsigned>(a.batch)), 256, 1, 0, 0,
                  true, s, G, a.rows, a.cols, a.ldg, a.stride_g, vec, pl.transposed, static_cast<const float*>(partial), parts, a.eps,
                  xh, xl, pl.np, pl.mp * pl.np, tiles_c);
}

}  // namespace

size_t ortho_workspace_size(int out_dtype, int64_t batch, int64_t rows, int64_t cols) {
    return plan_of(out_dtype, batch, rows, cols).total;
}

bool ortho_supports(int64_t batch, int64_t rows, int64_t cols) {
    const NsPlan pl = plan_of(DGA_F32, batch, rows, cols);
    const int64_t limit = (int64_t{1} << 31) - 256;  // rows and tiles are counted in 32 bits
    return batch <= 65535 && pl.np < limit && batch * pl.mp < limit && pl.mp / 64 * (pl.np / 64) * batch < limit;
}

cudaError_t ortho_launch(const OrthoArgs& a, const DeviceInfo& dev, int* launches) {
    const NsPlan pl = plan_of(a.out_dtype, a.batch, a.rows, a.cols);
    uint8_t* ws = static_cast<uint8_t*>(a.ws);
    float* partial = reinterpret_cast<float*>(ws);
    ws += round_up(a.batch * kMaxParts * 4, 256);
    __half *xh[2], *xl[2], *ah, *al, *bh, *bl;
    auto take = [&](size_t bytes) {
        __half* q = reinterpret_cast<__half*>(ws);
        ws += bytes;
        return q;
    };
    for (int i = 0; i < 2; ++i) {
        xh[i] = take(pl.x_bytes);
        xl[i] = take(pl.x_bytes);
    }
    ah = take(pl.a_bytes);
    bh = take(pl.a_bytes);
    al = pl.split ? take(pl.a_bytes) : nullptr;
    bl = pl.split ? take(pl.a_bytes) : nullptr;

    NsParams base{};
    base.split = pl.split;
    base.p_rows = base.q_rows = static_cast<uint32_t>(pl.mp);
    base.m = pl.m;
    base.n = pl.n;
    base.result = a.O;
    base.result_type = a.out_dtype;
    base.transposed = pl.transposed;
    const int64_t per16 = a.out_dtype == DGA_F32 ? 4 : 8;
    base.result_vec = aligned(a.O, 16) && a.ldo % per16 == 0 && (a.batch == 1 || a.stride_o % per16 == 0);
    // TMA writes the whole 16 bytes that a row's end lies in
    base.result_tma = base.result_vec && a.cols % per16 == 0;
    base.ldo = a.ldo;
    base.stride_o = a.stride_o;
    bool done = false;
    cudaError_t e = a.in_dtype == DGA_F32    ? launch_cluster<float>(a, pl, base, dev, &done)
                    : a.in_dtype == DGA_BF16 ? launch_cluster<__nv_bfloat16>(a, pl, base, dev, &done)
                                             : launch_cluster<__half>(a, pl, base, dev, &done);
    if (done) {
        *launches = 1;
        return e;
    }
    e = a.in_dtype == DGA_F32    ? launch_first<float>(a, pl, partial, xh[0], xl[0], dev, a.stream)
                    : a.in_dtype == DGA_BF16 ? launch_first<__nv_bfloat16>(a, pl, partial, xh[0], xl[0], dev, a.stream)
                                             : launch_first<__half>(a, pl, partial, xh[0], xl[0], dev, a.stream);
    if (e != cudaSuccess) return e;
    *launches += 2;

    // operand maps (128-row boxes K-major, 64-row ones the MN-major X) and value maps
    const int64_t all_rows = a.batch * pl.mp;
    struct Maps {
        CUtensorMap op, mn, value, mirror;
    } mx_h[2], mx_l[2], ma_h, ma_l, mb_h, mb_l;
    auto make = [&](Maps* m, const __half* base, int64_t ld, bool square) {
        if (e == cudaSuccess) e = half_map(&m->op, base, all_rows, ld, 128);
        if (e == cudaSuccess) e = value_map(&m->value, DGA_F16, base, ld, pl.mp, a.batch, ld, pl.mp * ld, true);
        if (e == cudaSuccess && square) e = value_map(&m->mirror, DGA_F16, base, ld, pl.mp, a.batch, ld, pl.mp * ld, false);
        if (e == cudaSuccess) e = half_map(&m->mn, base, all_rows, ld, 64);
    };
    for (int i = 0; i < 2; ++i) {
        make(&mx_h[i], xh[i], pl.np, false);
        make(&mx_l[i], xl[i], pl.np, false);
    }
    make(&ma_h, ah, pl.mp, true);
    make(&mb_h, bh, pl.mp, true);
    if (pl.split) {
        make(&ma_l, al, pl.mp, true);
        make(&mb_l, bl, pl.mp, true);
    } else {
        ma_l = ma_h;
        mb_l = mb_h;
    }
    CUtensorMap result = ma_h.value;  // not used without result_tma
    if (base.result_tma && e == cudaSuccess) {
        e = value_map(&result, a.out_dtype, a.O, a.cols, a.rows, a.batch, a.ldo, a.stride_o, !pl.transposed);
    }
    if (e != cudaSuccess) return e;

    for (int step = 0; step < a.steps; ++step) {
        const float ca = a.coefficients[3 * step], cb = a.coefficients[3 * step + 1], cc = a.coefficients[3 * step + 2];
        const int now = step & 1, next = now ^ 1;
        NsParams p = base;
        p.sym = 1;
        p.rows = p.ld = static_cast<int32_t>(pl.mp);
        p.out_lo = pl.split;
        NsMaps m;
        // A = X X^T
        p.num_kb = static_cast<uint32_t>(pl.np / 64);
        p.c_acc = 1.0f / kScale;
        m.p_h = m.q_h = mx_h[now].op;
        m.p_l = m.q_l = mx_l[now].op;
        m.q64_h = mx_h[now].mn;
        m.q64_l = mx_l[now].mn;
        m.old_h = m.old_l = ma_h.value;  // not used
        m.out_h = ma_h.value;
        m.out_l = ma_l.value;
        m.mirror_h = ma_h.mirror;
        m.mirror_l = ma_l.mirror;
        m.result = result;
        e = launch_product(p, m, a.batch, pl.mp, pl.mp, dev, a.stream);
        if (e != cudaSuccess) return e;
        // B = b A + c A^2
        p.num_kb = static_cast<uint32_t>(pl.mp / 64);
        p.c_old = cb;
        p.c_acc = cc / kScale;
        p.has_old = 1;
        p.old_lo = pl.split;
        m.p_h = m.q_h = ma_h.op;
        m.p_l = m.q_l = ma_l.op;
        m.q64_h = ma_h.mn;
        m.q64_l = ma_l.mn;
        m.old_l = ma_l.value;
        m.out_h = mb_h.value;
        m.out_l = mb_l.value;
        m.mirror_h = mb_h.mirror;
        m.mirror_l = mb_l.mirror;
        e = launch_product(p, m, a.batch, pl.mp, pl.mp, dev, a.stream);
        if (e != cudaSuccess) return e;
        // X <- a X + B X
        p.last = step + 1 == a.steps;
        p.sym = 0;
        p.q_mn = 1;
        p.ld = static_cast<int32_t>(pl.np);
        p.c_old = p.last ? ca / kScale : ca;
        p.c_acc = p.last ? 1.0f / (kScale * kScale) : 1.0f / kScale;
        p.old_lo = p.out_lo = 1;
        m.p_h = mb_h.op;
        m.p_l = mb_l.op;
        m.q_h = m.q64_h = mx_h[now].mn;
        m.q_l = m.q64_l = mx_l[now].mn;
        m.old_h = mx_h[now].value;
        m.old_l = mx_l[now].value;
        m.out_h = mx_h[next].value;
        m.out_l = mx_l[next].value;
        e = launch_product(p, m, a.batch, pl.mp, pl.np, dev, a.stream);
        if (e != cudaSuccess) return e;
        *launches += 3;
    }
    return cudaSuccess;
}

cudaError_t ns_status_take(int* status) {
    int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_ns_status, sizeof v);
    if (e != cudaSuccess) return e;
    if (v != 0) {
        int zero = 0;
        e = cudaMemcpyToSymbol(g_ns_status, &zero, sizeof zero);
    }
    *status = v;
    return e;
}

}  // namespace dga
