// mx_common.cuh -- the 4-bit microscaled matrices the mx kernels share.
//
// A matrix of R rows of K values is held as
//   codes   R rows of ld_codes bytes (a multiple of 16): value k of a row is
//           the E2M1 number (1 sign, 2 exponent, 1 mantissa bit: 0, 1/2, 1,
//           3/2, 2, 3, 4, 6) in byte k/2, bits 0-3 for even k and 4-7 for odd;
//   scales  one byte per block of 32 values (MXFP4: E8M0, the power of two
//           2^(byte - 127)) or 16 values (NVFP4: E4M3), tiled as the tensor
//           cores read them: 512-byte tiles of 128 rows x 4 blocks, the scale
//           of row r and block s at byte (r % 32) * 16 + (r / 32 % 4) * 4 +
//           s % 4 of tile (r / 128) * tiles_k + s / 4, tiles_k = ceil(blocks / 4);
//   and, optionally, one fp32 factor of the whole tensor.
// E2M1, E8M0 and the block of 32 are those of the OCP Microscaling Formats
// (MX) specification 1.0; E4M3 is that of the OCP 8-bit floating point
// specification.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "dga.h"

namespace dga {

constexpr int kMxTileBytes = 512;  // one scale tile

__host__ __device__ constexpr int mx_block(int format) { return format == DGA_MXFP4 ? 32 : 16; }

__host__ __device__ inline int64_t mx_tiles_k(int format, int64_t K) {
    const int64_t blocks = (K + mx_block(format) - 1) / mx_block(format);
    return (blocks + 3) / 4;
}

// Bytes of codes a row takes: K values, in whole groups of 32.
__host__ __device__ inline int64_t mx_row_bytes(int64_t K) { return (K + 31) / 32 * 16; }

// Byte offset of the scale of row r, block s.
__device__ __forceinline__ int64_t mx_scale_offset(int64_t r, int64_t s, int64_t tiles_k) {
    return ((r >> 7) * tiles_k + (s >> 2)) * kMxTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (s & 3);
}

}  // namespace dga
