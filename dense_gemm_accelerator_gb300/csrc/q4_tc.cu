// q4_tc.cu -- products of many rows with a 4-bit weight with group scales, and the
// gated layer on them, on the tensor cores with the weight read as its codes:
//     Y[M, N] = X[M, K] W^T + bias,  W = (q - z) s rounded to X's type.
//
// A weight value is two exact steps and one rounding away from its code: q - z is
// a small integer, exact in bf16 and fp16, and its product by s is rounded once,
// to X's type, which is what tcgen05.mma multiplies.  The sums are fp32.
//
// A CTA computes 128 weight rows (a gated layer's 128 gate rows and the 128 up
// rows that go with them, a second accumulator) by up to 256 (128) rows of X: the
// weight is the MMA's A, so an accumulator lane is an output column and a warp
// stores 32 consecutive outputs of a row of X whatever Y's alignment; the g and u
// of an output are in one lane.
//
//   warps 0-15   codes to values: a lane's row of 64 columns, 32 bytes of codes, into
//                the swizzled K-major rows that the MMA reads; teams of four warps
//                take the 64-column blocks in turn (gated: two teams the gate rows,
//                two the up rows).  After the loop they are the epilogue.
//   warps 16-19  scales and zero points, eight groups of each row at a time, as
//                words in shared memory (read group by group from the values'
//                warps, each load would touch 16 rows)
//   warp 20, 21  TMA: X in blocks of 64 columns, codes in blocks of 256
//   warp 22      MMA
//
// Where the tiles are fewer than the SMs, a cluster of up to eight CTAs shares a
// tile's K; their sums meet through distributed shared memory, each CTA adding
// a share of X's rows in the CTAs' order, so that results repeat.
//
// Bound by the values' warps and the MMA warp's issue beside them where X has few
// rows (8192 x 8192, bf16, groups of 128, 64 rows: 24 us, 1.5 TB/s of codes, where
// mma.sync on the codes takes 45), by the tensor cores where it has many (512 rows:
// 55 us, 1.24 PFLOP/s).  300 rows of 4099 x 4096: 19 us, 0.52 PFLOP/s, against 48
// through values written out first.
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

__device__ int g_q4_tc_status;  // non-zero: a bounded wait expired (role code)

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kValueWarps = 16, kScaleWarps = 4, kTeams = kValueWarps / 4;
constexpr int kXWarp = kValueWarps + kScaleWarps, kCodeWarp = kXWarp + 1, kMmaWarp = kXWarp + 2;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr uint32_t kMaxStages = 8, kMaxCodeStages = 4, kMaxSplits = 8;
constexpr uint32_t kATile = 128 * 128, kCodeTile = 128 * 128;  // 128 rows x 64 values, x 256 codes
constexpr uint32_t kPitch = 9;                                 // words of a row's eight groups in the table
constexpr uint32_t kMostSmem = 227 * 1024;
// full[8], empty[8], code full[4], code empty[4], table full[2], table empty[2], acc, drain, then tmem slot + abort flag
constexpr uint32_t kBarBytes = (2 * kMaxStages + 2 * kMaxCodeStages + 6) * 8 + 16;
enum : int { kRoleX = 1, kRoleCodes = 2, kRoleValues = 3, kRoleScales = 4, kRoleMma = 5, kRoleEpilogue = 6 };

struct Params {
    int64_t M, N, K;  // N: outputs (a gated layer's F)
    Q4Matrix q;
    const void* bias;
    void* Y;
    int64_t ldy;
    int act, shift;      // log2 of the group
    uint32_t tokens;     // rows of X in a tile, a multiple of 16
    uint32_t stages, stage_bytes, code_stages, ring_bytes, splits, code_blocks;
};

// Two neighbouring codes are a byte's halves, and two 16-bit numbers want them 16 bits
// apart: byte i of the codes goes to both halves of a word (bf16: the upper one from the
// codes shifted by one), where the lower code stands in the mantissa of kBoth as it is and
// the upper one 16 (8) times larger; a fused multiply-add takes that factor and the zero
// point off, exactly.  Nine integer steps to eight codes, which is what bounds the loop.
template <typename T> struct Value;
template <> struct Value<__nv_bfloat16> {
    using Two = __nv_bfloat162;
    static constexpr uint32_t kFmt = kFmtBF16;
    static constexpr uint32_t kBoth = 0x43004300u, kMask = 0x0078000fu;  // 128
    static constexpr uint32_t kFactors = 0x3e003f80u;                    // 1/8, 1
    // -(16 + z), -(128 + z)
    static __device__ __forceinline__ uint32_t offsets(uint32_t z) { return z * 0x00080001u + 0xc180c300u; }
    static __device__ __forceinline__ uint32_t upper(uint32_t w) { return w >> 1; }
};
template <> struct Value<__half> {
    using Two = __half2;
    static constexpr uint32_t kFmt = kFmtF16;
    static constexpr uint32_t kBoth = 0x64006400u, kMask = 0x00f0000fu;  // 1024
    static constexpr uint32_t kFactors = 0x2c003c00u;                    // 1/16, 1
    // -(64 + z), -(1024 + z)
    static __device__ __forceinline__ uint32_t offsets(uint32_t z) { return z * 0x00100001u + 0xd400e400u; }
    static __device__ __forceinline__ uint32_t upper(uint32_t w) { return w; }
};

// (q - z) s of the codes 2 i and 2 i + 1 of a word.
template <typename T, int i>
__device__ __forceinline__ uint32_t value2(uint32_t w, uint32_t upper, uint32_t offsets, uint32_t scale) {
    using V = Value<T>;
    const uint32_t code = (__byte_perm(w, upper, 0x4400 + 0x1111 * i) & V::kMask) | V::kBoth, factors = V::kFactors;
    typename V::Two c, f, o, s;
    memcpy(&c, &code, 4);
    memcpy(&f, &factors, 4);
    memcpy(&o, &offsets, 4);
    memcpy(&s, &scale, 4);
    c = __hmul2(__hfma2(c, f, o), s);
    uint32_t r;
    memcpy(&r, &c, 4);
    return r;
}

template <typename T>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t offsets, uint32_t scale) {
    const uint32_t u = Value<T>::upper(w);
    return make_uint4(value2<T, 0>(w, u, offsets, scale), value2<T, 1>(w, u, offsets, scale), value2<T, 2>(w, u, offsets, scale),
                      value2<T, 3>(w, u, offsets, scale));
}

// Zero from the n-th of eight values on (past K a scale that is no number would
// make one of X's zeros).
__device__ __forceinline__ uint4 first_of_8(uint4 v, int64_t n) {
    auto keep = [n](uint32_t w, int at) { return n > at + 1 ? w : n > at ? w & 0xffffu : 0u; };
    return make_uint4(keep(v.x, 0), keep(v.y, 2), keep(v.z, 4), keep(v.w, 6));
}

// True in one lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(is));
    return is != 0;
}

__device__ __forceinline__ void record_failure(int role, volatile int* abort_flag) {
    atomicCAS(&g_q4_tc_status, 0, role);
    *abort_flag = 1;
}

template <typename T>
__device__ __forceinline__ float activated(int act, float g) {
    switch (act) {
    case DGA_SILU: return act_value<DGA_SILU, true>(g);
    case DGA_GELU: return act_value<DGA_GELU, true>(g);
    case DGA_GELU_TANH: return act_value<DGA_GELU_TANH, true>(g);
    case DGA_RELU: return act_value<DGA_RELU, true>(g);
    default: return act_value<DGA_SIGMOID, true>(g);
    }
}

// kTiles: 1, or 2 for the gated layer; kShare: lanes to a row of 64 columns.
template <typename T, int kTiles, int kShare>
__global__ void __launch_bounds__(kThreads, 1)
    q4_tc_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmC, Params p) {
    using V = Value<T>;
    constexpr uint32_t kWriters = 4 * kTiles * kShare;  // warps that fill a stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* codes = smem + p.stages * p.stage_bytes;
    uint32_t* table = reinterpret_cast<uint32_t*>(smem + p.ring_bytes);
    constexpr uint32_t kTable = kTiles * 128 * kPitch;  // words of one of the two
    uint64_t* full = reinterpret_cast<uint64_t*>(table + 2 * kTable);
    uint64_t* empty = full + kMaxStages;
    uint64_t* code_full = empty + kMaxStages;
    uint64_t* code_empty = code_full + kMaxCodeStages;
    uint64_t* table_full = code_empty + kMaxCodeStages;
    uint64_t* table_empty = table_full + 2;
    uint64_t* acc = table_empty + 2;
    uint64_t* drain = acc + 1;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    // the same for the whole warp to the compiler's knowledge, too: descriptors then stay in
    // uniform registers (issued by a thread whose branch might diverge, a block's four MMAs
    // and their loop took 600 clocks beside the values' warps, which bound the kernel)
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = p.splits > 1 ? cluster_ctarank() : 0;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x / p.splits) * 128;
    const int64_t token0 = static_cast<int64_t>(blockIdx.y) * p.tokens;
    const uint32_t cb_begin = rank * p.code_blocks / p.splits, cb_end = (rank + 1) * p.code_blocks / p.splits;
    const uint32_t kb_begin = cb_begin * 4, kb_end = min(cb_end * 4, static_cast<uint32_t>((p.K + 63) / 64));
    const int log_blocks = p.shift - 5;  // 256-column blocks to eight groups
    bool ok = true;

    if (warp == kXWarp && lane == 0) {
        for (uint32_t s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], kWriters + 1);
            mbar_init(&empty[s], 1);
        }
        for (uint32_t s = 0; s < p.code_stages; ++s) {
            mbar_init(&code_full[s], 1);
            mbar_init(&code_empty[s], kValueWarps);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&table_full[b], kScaleWarps);
            mbar_init(&table_empty[b], kValueWarps);
        }
        mbar_init(acc, 1);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmC);
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (warp == kXWarp) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            for (uint32_t kb = kb_begin; kb < kb_end; ++kb) {
                if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleX, abort_flag);
                    __nanosleep(20000);  // let copies already issued land before teardown
                    break;
                }
                mbar_arrive_expect_tx(&full[stage], p.tokens * 128);
                tma_load_2d(smem + stage * p.stage_bytes + kTiles * kATile, &tmX, &full[stage], static_cast<int32_t>(kb * 64),
                            static_cast<int32_t>(token0));
                if (++stage == p.stages) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == kCodeWarp) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            for (uint32_t cb = cb_begin; cb < cb_end; ++cb) {
                if (!mbar_wait_bounded(&code_empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleCodes, abort_flag);
                    __nanosleep(20000);
                    break;
                }
                mbar_arrive_expect_tx(&code_full[stage], kTiles * kCodeTile);
                uint8_t* dst = codes + stage * (kTiles * kCodeTile);
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile)
                    tma_load_2d(dst + tile * kCodeTile, &tmC, &code_full[stage], static_cast<int32_t>(cb * 128),
                                static_cast<int32_t>(n0 + tile * p.N));
                if (++stage == p.code_stages) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == kMmaWarp) {
        const uint32_t idesc = idesc_mma(V::kFmt, 128, p.tokens);
        uint32_t stage = 0, phase = 0;
        for (uint32_t kb = kb_begin; kb < kb_end; ++kb) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[stage], phase, abort_flag, kWaitLimitNs))) {
                if (lane == 0) record_failure(kRoleMma, abort_flag);
                break;
            }
            tc_fence_after();
            const uint32_t addr = smem_u32(smem + stage * p.stage_bytes);
            const uint64_t x_desc = smem_desc_kmajor_sw128(addr + kTiles * kATile);
            if (elect_one()) {
#pragma unroll
                for (int tile = 0; tile < kTiles; ++tile) {
                    const uint64_t a_desc = smem_desc_kmajor_sw128(addr + tile * kATile);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma<V::kFmt>(tmem + tile * 128, a_desc + 2 * k, x_desc + 2 * k, idesc, (kb > kb_begin || k > 0) ? 1u : 0u);
                }
                tc_commit(&empty[stage]);
            }
            __syncwarp();
            if (++stage == p.stages) { stage = 0; phase ^= 1; }
        }
        if (elect_one()) {
            tc_commit(acc);
            tc_commit(drain);
        }
        __syncwarp();
        volatile int never = 0;
        mbar_wait_bounded(drain, 0, &never, kWaitLimitNs);
    } else if (warp >= kValueWarps) {
        // ------------------------------------------------ scales and zero points
        const uint16_t* scales = static_cast<const uint16_t*>(p.q.scales);
        const int64_t groups = (p.K + (1 << p.shift) - 1) >> p.shift;
        const uint32_t first = cb_begin >> log_blocks, last = (cb_end - 1) >> log_blocks;
        const int row0 = (warp - kValueWarps) * 32 * kTiles + (lane >> 3);
        for (uint32_t c = first, i = 0; c <= last; ++c, ++i) {
            if (!mbar_wait_bounded(&table_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
                if (lane == 0) record_failure(kRoleScales, abort_flag);
                break;
            }
            const int64_t group = static_cast<int64_t>(c) * 8 + (lane & 7), at = min(group, groups - 1);
            uint32_t* dst = table + (i & 1) * kTable + (lane & 7);
#pragma unroll
            for (int half = 0; half < kTiles; ++half) {
                uint32_t s[8], z[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    // loads without branches, so that they are in flight together
                    const int r = row0 + half * 32 + j * 4;
                    const int64_t row = min(n0 + (r & 127), p.N - 1) + (r >= 128 ? p.N : 0);
                    s[j] = __ldg(scales + row * p.q.ld_scales + at);
                    z[j] = 8;
                    if (p.q.zeros != nullptr) z[j] = __ldg(p.q.zeros + row * p.q.ld_zeros + at);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    dst[(row0 + half * 32 + j * 4) * kPitch] = ((group < groups ? s[j] : 0u) << 16) | (z[j] & 15u);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&table_full[i & 1]);
        }
    } else {
        // ------------------------------------------------ codes to values
        // a lane's row: eight lanes read, and write, eight different 16 bytes of the banks
        const int row = (warp & 3) * 32 + lane, tile = kTiles == 2 ? warp >> 3 : 0;
        const uint32_t swizzle = (lane & 7) << 4, line = row * 128;
        constexpr int kHalves = 2 / kShare;  // of a block's 64 columns
        const int first_half = kShare == 2 ? (warp >> 2) & 1 : 0;
        // Teams of four warps (eight: kShare) take the blocks in turn.  A wait for a stage
        // tells two phases apart, not three, so at block k a warp has to know that block
        // k - 2 stages has been multiplied: it learns at each block k that k - stages has
        // been, which is enough for its next one, k + kStep, with as many stages as teams.
        constexpr uint32_t kStep = kTeams / kTiles / kShare;
        const uint32_t team = (warp >> 2) / kShare % kStep;
        uint32_t stage = team, phase = 0, code_stage = 0, code_phase = 0, chunk = 0;
        while (stage >= p.stages) { stage -= p.stages; phase ^= 1; }
        for (uint32_t cb = cb_begin; ok && cb < cb_end; ++cb) {
            const bool enter = cb == cb_begin || (cb & ((1u << log_blocks) - 1)) == 0;
            const bool leave = ((cb + 1) & ((1u << log_blocks) - 1)) == 0;
            if ((enter && !mbar_wait_bounded(&table_full[chunk & 1], (chunk >> 1) & 1, abort_flag, kWaitLimitNs)) ||
                !mbar_wait_bounded(&code_full[code_stage], code_phase, abort_flag, kWaitLimitNs)) {
                ok = false;
                break;
            }
            const uint32_t code_line = smem_u32(codes + code_stage * (kTiles * kCodeTile) + tile * kCodeTile) + line + swizzle;
            const uint32_t* entries = table + (chunk & 1) * kTable + (tile * 128 + row) * kPitch;
#pragma unroll
            for (uint32_t j = 0; j < 4; j += kStep) {
                const uint32_t b = j + team, k0 = (cb * 4 + b) * 64;
                if (cb * 4 + b >= kb_end) break;
                uint4 w[kHalves];
                uint32_t offsets[kHalves], scale[kHalves];
#pragma unroll
                for (int i = 0; i < kHalves; ++i) {
                    const int h = first_half + i;
                    w[i] = ld_shared_v4(code_line ^ ((b * 2 + h) << 4));
                    const uint32_t entry = entries[((k0 + h * 32) >> p.shift) & 7];
                    offsets[i] = V::offsets(entry & 0xffffu);
                    scale[i] = __byte_perm(entry, 0, 0x3232);
                }
                const uint32_t dst = smem_u32(smem + stage * p.stage_bytes + tile * kATile) + line + swizzle;
                const bool last = k0 + 64 > p.K;
#pragma unroll
                for (int i = 0; i < kHalves; ++i) {
                    const int h = first_half + i;
                    uint4 v[4] = {values8<T>(w[i].x, offsets[i], scale[i]), values8<T>(w[i].y, offsets[i], scale[i]),
                                  values8<T>(w[i].z, offsets[i], scale[i]), values8<T>(w[i].w, offsets[i], scale[i])};
                    if (last) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) v[t] = first_of_8(v[t], p.K - k0 - h * 32 - t * 8);
                    }
                    // the first values are ready before the stage is waited for
                    if (i == 0 && !mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) st_shared_v4(dst ^ ((h * 4 + t) << 4), v[t]);
                }
                if (!ok) break;
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[stage]);
                stage += kStep;
                while (stage >= p.stages) { stage -= p.stages; phase ^= 1; }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&code_empty[code_stage]);
                if (leave) mbar_arrive(&table_empty[chunk & 1]);
            }
            if (leave) ++chunk;
            if (++code_stage == p.code_stages) { code_stage = 0; code_phase ^= 1; }
        }
        if (!ok && lane == 0) record_failure(kRoleValues, abort_flag);

        // ------------------------------------------------ results
        if (ok && !mbar_wait_bounded(acc, 0, abort_flag, kWaitLimitNs)) {
            if (lane == 0) record_failure(kRoleEpilogue, abort_flag);
            ok = false;
        }
        tc_fence_after();
        if (*abort_flag) ok = false;
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok);
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int64_t n = n0 + (warp & 3) * 32 + lane;
        const T* bias = static_cast<const T*>(p.bias);
        const bool in = n < p.N;
        float b[kTiles];
#pragma unroll
        for (int t = 0; t < kTiles; ++t) b[t] = bias != nullptr && in ? OutT<T>::load(bias + n + t * p.N) : 0.0f;
        auto store = [&](uint32_t token, const float (&v)[kTiles]) {
            if (!in || token0 + token >= p.M) return;
            float y = v[0] + b[0];
            if constexpr (kTiles == 2) y = activated<T>(p.act, y) * (v[1] + b[1]);
            OutT<T>::store(static_cast<T*>(p.Y) + (token0 + token) * p.ldy + n, y);
        };
        // 16 rows of X at a time, dealt to the four warps of a quarter of the lanes
        for (uint32_t t0 = (warp >> 2) * 16; ok && t0 < p.tokens; t0 += kValueWarps / 4 * 16) {
            uint32_t r[kTiles][16];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) tmem_ld_32x32b_x16(tmem + lanes + t * 128 + t0, r[t]);
            tmem_ld_wait();
            if (p.splits == 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float v[kTiles];
#pragma unroll
                    for (int t = 0; t < kTiles; ++t) v[t] = __uint_as_float(r[t][j]);
                    store(t0 + j, v);
                }
            } else {
                // every copy has landed and every MMA read it: [tile][row of X][weight row] over the rings
#pragma unroll
                for (int t = 0; t < kTiles; ++t)
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        st_shared_u32(smem_u32(smem) + ((t * p.tokens + t0 + j) * 128 + (warp & 3) * 32 + lane) * 4, r[t][j]);
            }
        }
        if (p.splits > 1) {
            __syncwarp();
            cluster_sync();
            const uint32_t begin = rank * p.tokens / p.splits, end = (rank + 1) * p.tokens / p.splits;
            for (uint32_t token = begin + (warp >> 2); ok && token < end; token += kValueWarps / 4) {
                float v[kTiles];
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    const uint32_t at = smem_u32(smem) + ((t * p.tokens + token) * 128 + (warp & 3) * 32 + lane) * 4;
                    float part[kMaxSplits];
#pragma unroll
                    for (uint32_t s = 0; s < kMaxSplits; ++s)
                        part[s] = s < p.splits ? ld_shared_cluster_f32(map_to_cta(at, s)) : 0.0f;
                    v[t] = part[0];
#pragma unroll
                    for (uint32_t s = 1; s < kMaxSplits; ++s)
                        if (s < p.splits) v[t] += part[s];
                }
                store(token, v);
            }
        }
    }

    __syncwarp();
    if (p.splits > 1) {
        if (warp >= kValueWarps) cluster_sync();  // the one in which sums are ready
        cluster_sync();                           // none leaves while another reads its sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 256);
    }
}

// ---- host side -----------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t make_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, int64_t rows, int64_t cols, int64_t row_bytes,
                     uint32_t box_cols, uint32_t box_rows) {
    const EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row_bytes)};
    const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
    return encode(map, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// Shared memory: two tables, barriers, alignment; a stage; the stages that fit.
template <int kTiles> constexpr uint32_t kFixedBytes = 2 * kTiles * 128 * kPitch * 4 + kBarBytes + 1024;
template <int kTiles> constexpr uint32_t kCodeStages = kTiles == 1 ? 3 : 2;
template <int kTiles> uint32_t stage_bytes(uint32_t tokens) { return kTiles * kATile + tokens * 128; }
template <int kTiles> uint32_t stages(uint32_t tokens) {
    return std::min(kMaxStages, (kMostSmem - kFixedBytes<kTiles> - kCodeStages<kTiles> * kTiles * kCodeTile) / stage_bytes<kTiles>(tokens));
}

template <typename T, int kTiles, int kShare>
cudaError_t launch_shared(const CUtensorMap& x, const CUtensorMap& c, Params p, int64_t row_tiles, int64_t token_tiles, cudaStream_t s) {
    auto kern = q4_tc_kernel<T, kTiles, kShare>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostSmem));
    if (e != cudaSuccess) return e;
    p.code_stages = kCodeStages<kTiles>;
    p.stage_bytes = stage_bytes<kTiles>(p.tokens);
    p.stages = stages<kTiles>(p.tokens);
    p.ring_bytes = p.stages * p.stage_bytes + p.code_stages * kTiles * kCodeTile;
    // a stage to each team (see the kernel), and room for a tile's sums
    if (p.stages < kTeams / kTiles / kShare || p.tokens * 512 * kTiles > p.ring_bytes) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(row_tiles * p.splits), static_cast<unsigned>(token_tiles));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = p.ring_bytes + kFixedBytes<kTiles>;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, x, c, p);
}

// Two lanes to a row where the stages are fewer than the teams (more than 207 rows of X).
template <typename T>
cudaError_t launch(const CUtensorMap& x, const CUtensorMap& c, const Params& p, bool gated, int64_t row_tiles, int64_t token_tiles, cudaStream_t s) {
    if (gated) return launch_shared<T, 2, 1>(x, c, p, row_tiles, token_tiles, s);
    return stages<1>(p.tokens) >= kTeams ? launch_shared<T, 1, 1>(x, c, p, row_tiles, token_tiles, s)
                                         : launch_shared<T, 1, 2>(x, c, p, row_tiles, token_tiles, s);
}

}  // namespace

cudaError_t q4_tc_launch(int dtype, int act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const Q4Matrix& q,
                         const void* bias, void* Y, int64_t ldy, bool gated, const DeviceInfo& dev, cudaStream_t stream) {
    Params p{};
    p.M = M, p.N = N, p.K = K;
    p.q = q;
    p.bias = bias;
    p.Y = Y, p.ldy = ldy;
    p.act = act;
    p.shift = q.group == 32 ? 5 : q.group == 64 ? 6 : 7;
    const int64_t most = gated ? 128 : 256;
    const int64_t token_tiles = (M + most - 1) / most, row_tiles = (N + 127) / 128;
    p.tokens = static_cast<uint32_t>(((M + token_tiles - 1) / token_tiles + 15) / 16 * 16);
    p.code_blocks = static_cast<uint32_t>((K + 255) / 256);
    // as many parts of K as leave each a CTA on an SM of its own, and two blocks of codes
    p.splits = static_cast<uint32_t>(std::max<int64_t>(
        1, std::min<int64_t>({kMaxSplits, dev.sm_count / (token_tiles * row_tiles), p.code_blocks / 2})));
    if (row_tiles * p.splits > 0x7fffffff || token_tiles > 65535) return cudaErrorInvalidConfiguration;
    CUtensorMap x, c;
    cudaError_t e = make_map(&x, CU_TENSOR_MAP_DATA_TYPE_UINT16, X, M, K, ldx * 2, 64, p.tokens);
    if (e == cudaSuccess) e = make_map(&c, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, gated ? 2 * N : N, mx_row_bytes(K), q.ld, 128, 128);
    if (e != cudaSuccess) return e;
    return dtype == DGA_BF16 ? launch<__nv_bfloat16>(x, c, p, gated, row_tiles, token_tiles, stream)
                             : launch<__half>(x, c, p, gated, row_tiles, token_tiles, stream);
}

cudaError_t q4_tc_status_take(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_q4_tc_status, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_q4_tc_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace dga
