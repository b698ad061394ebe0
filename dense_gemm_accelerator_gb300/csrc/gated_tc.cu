// gated_tc.cu -- the gated feed-forward layer on the tensor cores,
//     [g | u] = X W^T + b,  H = act(g) * u,   bf16 or fp16, fp32 sums,
// both products, the activation and the product in one kernel; where the layer is
// trained it also writes P = [g | u].
//
// A cluster of two CTAs computes 256 rows of X by 128 columns of H with
// tcgen05.mma.cta_group::2 (M = 256, N = 256, K = 16).  The MMA's N is the CTAs'
// B operands side by side, so the even CTA loads the 128 gate rows of W and the
// odd one the 128 up rows that go with them: columns c and 128 + c of the
// accumulator are the g and u of column c of H, in the same lane, and the product
// needs no exchange.  For the tensor cores the layer is then the product X W^T as
// it stands, and the epilogue, which runs beside the next tile's MMAs out of two
// accumulators, writes a third of what P alone would take.
//
//   warp 0      TMA producer (both CTAs): boxes of 128 rows x 64 columns of X and
//               W, 128-byte swizzle, a ring of six stages; every copy counts on the
//               even CTA's barrier
//   warp 1      MMA issuer (even CTA)
//   warps 2-9   epilogue: two per quarter of the accumulator's rows, each 64 of the
//               128 column pairs, 32 at a time; results leave by TMA from 32 x 32
//               boxes (rows of 64 bytes, swizzled), or, where their rows are not
//               whole 16 bytes apart, transposed through the same memory, a row of
//               32 values to a store
//
// Bound by the tensor cores where there are many rows.  Up to 256 rows the tiles are the
// ceil(F / 128) of one tile row, each on two SMs that walk all of K alone, with MMAs of
// 256 rows whatever X has: K = 8192 takes 41 us for F = 1024 (32 rows or 200; the tensor
// pipe of the 16 SMs at work 80 % busy), 2048 and 4096 alike, where W's bytes take 5, 10
// and 20.  4096 to 4096, 32 rows: 24.4 us, W's bytes 10.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "dga_internal.h"
#include "epilogue.cuh"
#include "gated_act.cuh"
#include "ptx.cuh"

namespace dga {

__device__ int g_gated_status;  // non-zero: a bounded wait expired (role code)

namespace {

constexpr uint64_t kWaitLimitNs = 4000000000ull;  // 4 s
constexpr int kStages = 6, kEpiWarps = 8, kThreads = (2 + kEpiWarps) * 32;
constexpr uint32_t kOperand = 128 * 128, kStage = 2 * kOperand;
constexpr uint32_t kBox = 32 * 64, kEpiWarpBytes = 2 * kBox;
constexpr uint32_t kEpi = kStages * kStage, kBar = kEpi + kEpiWarps * kEpiWarpBytes;
// full[S], empty[S], acc_full[2], acc_empty[2], drain, then tmem slot + abort flag
constexpr uint32_t kLaunchBytes = kBar + (2 * kStages + 5) * 8 + 16 + 1024;
enum : int { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3 };

struct Params {
    int64_t M, F;
    const void* bias;
    void* H;
    int64_t ldh;
    void* P;
    int64_t ldp;
    int act;
    uint32_t tiles_m, tiles_n, num_tiles, num_kb, group_m;
    uint32_t tma_h, tma_p;  // results that TMA can store
};

__device__ __forceinline__ void record_failure(int role, volatile int* abort_flag) {
    atomicCAS(&g_gated_status, 0, role);
    *abort_flag = 1;
}

// Tiles in groups of group_m tile rows, whose panels of X stay in L2 while W's
// pass by.
__device__ __forceinline__ void tile_coords(uint32_t t, const Params& p, uint32_t& tm, uint32_t& tn) {
    const uint32_t group_size = p.group_m * p.tiles_n;
    const uint32_t group = t / group_size, first_m = group * p.group_m;
    const uint32_t gm = min(p.tiles_m - first_m, p.group_m), r = t % group_size;
    tm = first_m + r % gm;
    tn = r / gm;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    T two[2];
    OutT<T>::store(&two[0], a);
    OutT<T>::store(&two[1], b);
    uint32_t w;
    memcpy(&w, two, 4);
    return w;
}

// 32 values of this lane's row to columns col .. col + 31 of an output.
template <typename T>
__device__ __forceinline__ void store_32(const CUtensorMap* map, uint32_t by_tma, T* out, int64_t ld, uint8_t* boxes, int lane, int64_t row,
                                         int64_t col, int64_t M, int64_t F, const float (&v)[32], uint32_t& turn) {
    if (by_tma) {
        uint8_t* box = boxes + (turn & 1) * kBox;
        if (lane == 0) bulk_wait_read<1>();  // the store before last has read this box
        __syncwarp();
        // rows of 64 bytes, two to a line of 128: pieces of 16 swizzled by the line
#pragma unroll
        for (int q = 0; q < 4; ++q)
            st_shared_v4(smem_u32(box) + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4),
                         make_uint4(pack2<T>(v[q * 8], v[q * 8 + 1]), pack2<T>(v[q * 8 + 2], v[q * 8 + 3]),
                                    pack2<T>(v[q * 8 + 4], v[q * 8 + 5]), pack2<T>(v[q * 8 + 6], v[q * 8 + 7])));
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (row < M && col < F) tma_store_2d(map, box, static_cast<int32_t>(col), static_cast<int32_t>(row));
            bulk_commit();
        }
        ++turn;
    } else {
        // element (row, c) at word row * 32 + (c + row) % 32: neither direction meets in a bank
        if (lane == 0) bulk_wait_read<0>();  // stores of the other output that still read the boxes
        __syncwarp();
        const uint32_t words = smem_u32(boxes);
#pragma unroll
        for (int c = 0; c < 32; ++c) st_shared_u32(words + (lane * 32 + ((c + lane) & 31)) * 4, __float_as_uint(v[c]));
        __syncwarp();
        const int rows = static_cast<int>(min(static_cast<int64_t>(32), M - row));
        T* dst = out + row * ld + col + lane;
        const bool in = col + lane < F;
#pragma unroll 8
        for (int i = 0; i < 32; ++i, dst += ld)
            if (in && i < rows) OutT<T>::store(dst, ld_shared_f32(words + (i * 32 + ((lane + i) & 31)) * 4));
        __syncwarp();
    }
}

template <int kAct>
__device__ __forceinline__ void multiply(float (&h)[32], const float (&g)[32], const float (&u)[32]) {
#pragma unroll
    for (int c = 0; c < 32; ++c) h[c] = act_value<kAct, true>(g[c]) * u[c];
}

template <uint32_t kFmt, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    gated_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmH, const __grid_constant__ CUtensorMap tmG,
                      const __grid_constant__ CUtensorMap tmU, Params p) {
    constexpr uint32_t kIdesc = idesc_mma(kFmt, 256, 256);
    constexpr uint16_t kBothCtas = 0x3;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBar);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);  // one lane of each epilogue warp of both CTAs
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmW);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // barriers of both CTAs initialised before any remote arrive
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
                const int32_t x_row = static_cast<int32_t>(tm * 256 + rank * 128);
                const int32_t w_row = static_cast<int32_t>(tn * 128 + (leader ? 0 : p.F));
                for (uint32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait_bounded<true>(&empty[stage], phase ^ 1, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleProducer, abort_flag);
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + stage * kStage;
                    if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStage);
                    const uint32_t bar = map_to_cta(smem_u32(&full[stage]), 0);
                    tma_load_2d_pair(dst, &tmX, bar, static_cast<int32_t>(kb * 64), x_row);
                    tma_load_2d_pair(dst + kOperand, &tmW, bar, static_cast<int32_t>(kb * 64), w_row);
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                }
            }
            if (!ok) __nanosleep(20000);  // let copies already issued land before teardown
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            uint32_t stage = 0, phase = 0, i = 0;
            bool ok = true;
            for (uint32_t t = cluster_id; ok && t < p.num_tiles; t += n_clusters, ++i) {
                if (!mbar_wait_bounded<true>(&acc_empty[i & 1], ((i >> 1) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
                    record_failure(kRoleMma, abort_flag);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + (i & 1) * 256;
                for (uint32_t kb = 0; kb < p.num_kb; ++kb) {
                    if (!mbar_wait_bounded<true>(&full[stage], phase, abort_flag, kWaitLimitNs)) {
                        record_failure(kRoleMma, abort_flag);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t addr = smem_u32(smem + stage * kStage);
                    const uint64_t a_desc = smem_desc_kmajor_sw128(addr), b_desc = smem_desc_kmajor_sw128(addr + kOperand);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc_mma_pair<kFmt>(d, a_desc + 2 * k, b_desc + 2 * k, kIdesc, (kb > 0 || k > 0) ? 1u : 0u);
                    tc_commit_pair_multicast(&empty[stage], kBothCtas);
                    if (++stage == kStages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                tc_commit_pair_multicast(&acc_full[i & 1], kBothCtas);
            }
            tc_commit_pair_multicast(drain, 0x1);
            volatile int never = 0;
            mbar_wait_bounded(drain, 0, &never, kWaitLimitNs);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t* boxes = smem + kEpi + (warp - 2) * kEpiWarpBytes;
        const T* bias = static_cast<const T*>(p.bias);
        uint32_t i = 0, turn = 0;
        for (uint32_t t = cluster_id; t < p.num_tiles; t += n_clusters, ++i) {
            uint32_t tm, tn;
            tile_coords(t, p, tm, tn);
            const int64_t row = static_cast<int64_t>(tm) * 256 + rank * 128 + quarter * 32;
            if (!mbar_wait_bounded<true>(&acc_full[i & 1], (i >> 1) & 1, abort_flag, kWaitLimitNs)) {
                record_failure(kRoleEpilogue, abort_flag);
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
                const int at = half * 64 + c * 32;
                const int64_t col = static_cast<int64_t>(tn) * 128 + at;
                uint32_t r[2][32];
                tmem_ld_32x32b_x32(tmem + lane_base + (i & 1) * 256 + at, r[0]);
                tmem_ld_32x32b_x32(tmem + lane_base + (i & 1) * 256 + 128 + at, r[1]);
                tmem_ld_wait();
                if (c == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_signal_cluster(map_to_cta(smem_u32(&acc_empty[i & 1]), 0));
                }
                float g[32], u[32], h[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) g[j] = __uint_as_float(r[0][j]), u[j] = __uint_as_float(r[1][j]);
                if (bias != nullptr) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (col + j < p.F) {
                            g[j] += OutT<T>::load(bias + col + j);
                            u[j] += OutT<T>::load(bias + p.F + col + j);
                        }
                }
                if (p.P != nullptr) {
                    store_32<T>(&tmG, p.tma_p, static_cast<T*>(p.P), p.ldp, boxes, lane, row, col, p.M, p.F, g, turn);
                    store_32<T>(&tmU, p.tma_p, static_cast<T*>(p.P) + p.F, p.ldp, boxes, lane, row, col, p.M, p.F, u, turn);
                }
                switch (p.act) {
                case DGA_SILU: multiply<DGA_SILU>(h, g, u); break;
                case DGA_GELU: multiply<DGA_GELU>(h, g, u); break;
                case DGA_GELU_TANH: multiply<DGA_GELU_TANH>(h, g, u); break;
                case DGA_RELU: multiply<DGA_RELU>(h, g, u); break;
                default: multiply<DGA_SIGMOID>(h, g, u); break;
                }
                store_32<T>(&tmH, p.tma_h, static_cast<T*>(p.H), p.ldh, boxes, lane, row, col, p.M, p.F, h, turn);
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

// ---- host side -----------------------------------------------------------------------

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                   const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t make_map(CUtensorMap* map, bool bf16, const void* base, int64_t rows, int64_t cols, int64_t ld, uint32_t box_cols,
                     uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
                  strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <uint32_t kFmt, typename T>
cudaError_t launch_pair(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& h, const CUtensorMap& g,
                        const CUtensorMap& u, const Params& p,
                        const DeviceInfo& dev, cudaStream_t s) {
    auto kern = gated_pair_kernel<kFmt, T>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kLaunchBytes));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kLaunchBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    // clusters of two that fit at once (queried once per kernel and device)
    static int cached[64] = {};
    static std::mutex mu;
    int clusters = dev.sm_count / 2;
    {
        std::lock_guard<std::mutex> lock(mu);
        const bool known = dev.ordinal >= 0 && dev.ordinal < 64;
        if (known && cached[dev.ordinal] > 0) {
            clusters = cached[dev.ordinal];
        } else {
            cfg.gridDim = dim3(2 * clusters);
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0) clusters = n;
            else cudaGetLastError();
            if (known) cached[dev.ordinal] = clusters;
        }
    }
    cfg.gridDim = dim3(2 * std::min<uint32_t>(p.num_tiles, static_cast<uint32_t>(std::max(clusters, 1))));
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, x, w, h, g, u, p);
}

}  // namespace

bool gated_tc_supports(const GatedArgs& a) {
    return a.dtype != DGA_F32 && a.K >= 1 && a.ldx % 8 == 0 && a.ldw % 8 == 0 && aligned(a.X, 16) && aligned(a.W, 16) &&
           tensor_map_encoder() != nullptr;
}

cudaError_t gated_tc_launch(const GatedArgs& a, const DeviceInfo& dev) {
    const bool bf16 = a.dtype == DGA_BF16;
    Params p{};
    p.M = a.M, p.F = a.F;
    p.bias = a.bias;
    p.H = a.H, p.ldh = a.ldh;
    p.P = a.P, p.ldp = a.ldp;
    p.act = a.act;
    p.tiles_m = static_cast<uint32_t>((a.M + 255) / 256);
    p.tiles_n = static_cast<uint32_t>((a.F + 127) / 128);
    if (static_cast<uint64_t>(p.tiles_m) * p.tiles_n >= (uint64_t{1} << 31)) return cudaErrorInvalidConfiguration;
    p.num_tiles = p.tiles_m * p.tiles_n;
    p.num_kb = static_cast<uint32_t>((a.K + 63) / 64);
    // the panels of X of a group, 32 MB of them
    const double panel = 256.0 * static_cast<double>(a.K) * 2;
    p.group_m = std::min(p.tiles_m, std::max(8u, std::min(64u, static_cast<uint32_t>(32.0 * 1024 * 1024 / panel))));
    // TMA leaves out what lies past a row's end by 16 bytes at a time
    p.tma_h = aligned(a.H, 16) && a.ldh % 8 == 0 && a.F % 8 == 0;
    p.tma_p = a.P != nullptr && aligned(a.P, 16) && a.ldp % 8 == 0 && a.F % 8 == 0;
    CUtensorMap x, w, h{}, g{}, u{};  // g, u: P's halves, each with its own right edge
    cudaError_t e = make_map(&x, bf16, a.X, a.M, a.K, a.ldx, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess) e = make_map(&w, bf16, a.W, 2 * a.F, a.K, a.ldw, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess && p.tma_h) e = make_map(&h, bf16, a.H, a.M, a.F, a.ldh, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e == cudaSuccess && p.tma_p) e = make_map(&g, bf16, a.P, a.M, a.F, a.ldp, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e == cudaSuccess && p.tma_p)
        e = make_map(&u, bf16, static_cast<const uint16_t*>(a.P) + a.F, a.M, a.F, a.ldp, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e != cudaSuccess) return e;
    return bf16 ? launch_pair<kFmtBF16, __nv_bfloat16>(x, w, h, g, u, p, dev, a.stream)
                : launch_pair<kFmtF16, __half>(x, w, h, g, u, p, dev, a.stream);
}

cudaError_t gated_status_take(int* status) {
    int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_gated_status, sizeof v);
    if (e == cudaSuccess && v != 0) e = cudaMemcpyToSymbol(g_gated_status, &zero, sizeof zero);
    *status = v;
    return e;
}

}  // namespace dga
