// q4_rows_f16.cu -- the fp16 kernels of q4_rows.cuh.
#include "q4_rows.cuh"

namespace dga {

cudaError_t q4rows::launch_f16(const CUtensorMap& tm, const CUtensorMap& tmX, const CUtensorMap& tmTail, const Params& p, int tiles, unsigned blocks, cudaStream_t s) {
    return launch_type<__half>(tm, tmX, tmTail, p, tiles, blocks, s);
}

cudaError_t q4rows::take_status_f16(int* status) { return take_status(status); }

}  // namespace dga
