// hqq_decode.cu -- the weight-only linear layer for few tokens (hqq_decode.cuh).
#include "hqq_decode.cuh"

namespace hqq {

cudaError_t launch_decode(const LinearParams& p, const void* X, int nbits, int64_t packed_bytes,
                          cudaStream_t stream) {
    return launch_few<false>(p, LowRankEpi{}, X, nbits, packed_bytes, stream);
}

}  // namespace hqq
