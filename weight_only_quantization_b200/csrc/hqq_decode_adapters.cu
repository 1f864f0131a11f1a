// hqq_decode_adapters.cu -- the linear layer with the tokens' adapters, few tokens
// (hqq_decode.cuh with the low-rank term added before the rounding).
#include "hqq_decode.cuh"

namespace hqq {

cudaError_t launch_decode_adapters(const LinearParams& p, const LowRankEpi& lr, const void* X,
                                   int nbits, int64_t packed_bytes, cudaStream_t stream) {
    return launch_few<true>(p, lr, X, nbits, packed_bytes, stream);
}

}  // namespace hqq
