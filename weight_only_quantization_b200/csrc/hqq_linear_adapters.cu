// hqq_linear_adapters.cu -- Y = X W_hat^T + the tokens' adapters, many tokens
// (hqq_linear.cuh with the low-rank term added in its epilogue).
#include "hqq_linear.cuh"

namespace hqq {

cudaError_t launch_linear_adapters(const LinearParams& prm, const LowRankEpi& lr, const void* X,
                                   int nbits, cudaStream_t stream) {
    return launch_mode<kAdapters>(prm, lr, X, prm.K, nbits, stream);
}

}  // namespace hqq
