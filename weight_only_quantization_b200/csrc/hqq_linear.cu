// hqq_linear.cu -- Y = X W_hat^T, the weight-only linear layer (hqq_linear.cuh).
#include "hqq_linear.cuh"

namespace hqq {

cudaError_t launch_linear(const LinearParams& prm, const void* X, int nbits, cudaStream_t stream) {
    return launch_mode<kPlain>(prm, LowRankEpi{}, X, prm.K, nbits, stream);
}

}  // namespace hqq
