// hqq_adapters.cuh -- launch parameters of the low-rank adapters' own kernels
// (hqq_adapters.cu).
#pragma once
#include "hqq_params.cuh"

namespace hqq {

// T[m, j] = s_a sum_k X[m, k] F[a, k, j] for the tokens that have an adapter.
struct ShrinkParams {
    const __half* X;          // [M, K], rows ldx apart (a multiple of 8), 16-byte aligned;
                              // columns K .. ldx - 1 hold zeros
    const void* F;            // element (a, k, j) at a * sa + k * sk + j * sj
    const int32_t* index;     // NULL: adapter 0 for every token
    const float* scaling;     // NULL: 1
    float* T;                 // [M, ld]
    const int32_t* order;     // NULL, or the tokens sorted by adapter ..
    const int32_t* start;     // .. and where each adapter's begin (start[count]: all)
    int64_t M, K, ldx, sa, sk, sj;
    int ld, rank, count, dtype;
    int beside;               // may run beside the kernel launched before it
};

// dA[a, j, k] and dB[a, n, j] from scaled P = dY B and T = X A^T.
struct FactorGradParams {
    const __half* X;          // [M, K], rows ldx apart
    const __half* dY;         // [M, N], rows ldy apart (a multiple of 8; zeros behind N)
    const float* P;           // [M, ld]
    const float* T;
    const int32_t* order;     // NULL: every token has adapter 0
    const int32_t* start;
    float* dA;                // nullable
    float* dB;                // nullable
    int64_t M, N, K, ldx, ldy;
    int ld, rank, count, tiles_a;
};

}  // namespace hqq
