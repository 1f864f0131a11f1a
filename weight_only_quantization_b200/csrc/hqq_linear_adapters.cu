// hqq_linear_adapters.cu -- Y = X W_hat^T + the tokens' adapters, many tokens
// (hqq_gemm.cuh).
#include "hqq_gemm.cuh"

namespace hqq {

cudaError_t launch_linear_adapters(const LinearParams& prm, const LowRankEpi& lr, const void* X,
                                   int nbits, cudaStream_t stream) {
    return launch_gemm<false>(prm, lr, X, prm.K, nbits, stream);
}

}  // namespace hqq
