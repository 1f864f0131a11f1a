// hqq_linear_backward.cu -- dX = dY W_hat (+ the adapters' term), the input
// gradient of the weight-only linear layer (hqq_gemm.cuh, transposed weights).
#include "hqq_gemm.cuh"

namespace hqq {

// dY: fp16 [M, N], rows ld values apart (a multiple of 8), 16-byte aligned;
// prm.Y is dX [M, K]; lr.T == NULL leaves the adapters out.
cudaError_t launch_linear_backward(const LinearParams& prm, const LowRankEpi& lr, const void* dY,
                                   int64_t ld, int nbits, cudaStream_t stream) {
    return launch_gemm<true>(prm, lr, dY, ld, nbits, stream);
}

}  // namespace hqq
