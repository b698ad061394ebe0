// q4_rows.cu -- the host side of q4_rows.cuh and its bf16 kernels.
#include "q4_rows.cuh"

namespace dga {

cudaError_t q4rows::launch_bf16(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s) {
    return launch_type<__nv_bfloat16>(tm, tmX, tmTail, p, tiles, blocks, s);
}

cudaError_t q4_rows_launch(int dtype, int act, int64_t M, int64_t N, int64_t K, const void* X, int64_t ldx, const Q4Matrix& q,
                           const void* bias, void* Y, int64_t ldy, bool gated, const DeviceInfo& dev, cudaStream_t stream) {
    using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                       const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                       CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    const EncodeTiledFn encode = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
    if (!encode) return cudaErrorNotSupported;
    q4rows::Params p{};
    p.M = M, p.N = N, p.K = K;
    p.q = q;
    p.bias = bias;
    p.Y = Y, p.ldy = ldy;
    p.act = act;
    p.gated = gated;
    p.table_vec = aligned(q.scales, 16) && q.ld_scales % 8 == 0 && (!q.zeros || (aligned(q.zeros, 8) && q.ld_zeros % 8 == 0));
    p.shift = q.group == 32 ? 5 : q.group == 64 ? 6 : 7;
    // whole waves of one block per SM, as few as keep every block at the most rows
    // it can have, but no more blocks than tiles of 16
    const int64_t most = gated ? 32 : 64;
    const int64_t least = (N + most - 1) / most, waves = (least + dev.sm_count - 1) / dev.sm_count;
    const int64_t blocks = std::min(waves * dev.sm_count, (N + 15) / 16);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    p.box_rows = static_cast<uint32_t>((N + blocks - 1) / blocks);
    const uint32_t rows = p.box_rows;
    const int tiles = gated ? (rows <= 16 ? 2 : 4) : (rows <= 16 ? 1 : rows <= 32 ? 2 : 4);
    const int64_t total = gated ? 2 * N : N;
    CUtensorMap tm, tmX{}, tmTail{};
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(mx_row_bytes(K)), static_cast<cuuint64_t>(total)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(q.ld)};
    const cuuint32_t box[2] = {128, rows};
    const cuuint32_t one[2] = {1, 1};
    if (encode(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q.codes), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    {
        // X: whole lines of 64 columns, and by columns for the stage that K ends in
        const cuuint64_t xdims[3] = {64, static_cast<cuuint64_t>(M), static_cast<cuuint64_t>(K / 64)};
        const cuuint64_t xstrides[2] = {static_cast<cuuint64_t>(ldx) * 2, 128};
        const cuuint64_t tdims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(M)};
        const cuuint32_t stage_k = q4rows::stage_columns(M);
        const cuuint32_t xbox[3] = {64, static_cast<cuuint32_t>(M), stage_k / 64};
        const cuuint32_t ones[3] = {1, 1, 1};
        if (K >= stage_k &&
            encode(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(X), xdims, xstrides, xbox, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
        if (K % stage_k != 0 &&
            encode(&tmTail, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(X), tdims, xstrides, xbox, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    return dtype == DGA_BF16 ? q4rows::launch_bf16(tm, tmX, tmTail, p, tiles, static_cast<unsigned>(blocks), stream)
                             : q4rows::launch_f16(tm, tmX, tmTail, p, tiles, static_cast<unsigned>(blocks), stream);
}

cudaError_t q4_status_take(int* status) {
    int f16 = 0;
    cudaError_t e = q4rows::take_status(status);
    if (e == cudaSuccess) e = q4rows::take_status_f16(&f16);
    if (f16 != 0) *status = f16;
    return e;
}

}  // namespace dga
