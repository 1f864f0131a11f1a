// hqq_lowrank_epi.cuh -- the low-rank term that the linear-layer kernels add to
// their fp32 sums: for token m with adapter a and output feature f
//   sum_j T[m, j] * F[a, f, j],
// T [M, ld] fp32 already scaled (hqq_adapters.cu), ld = the rank rounded up to 16
// with zeros behind it; F is the adapters' second factor (B for the layer, A for
// its input gradient) in fp16, bf16 or fp32, addressed by strides.  The sum runs
// over j in fp32 fused multiply-adds.  A token without an adapter is skipped
// (its row of T is never read).
#pragma once
#include <cuda_bf16.h>

#include "hqq_params.cuh"

namespace hqq {

struct LowRankEpi {
    const float* T;          // NULL: no term
    const int32_t* index;    // NULL: adapter 0 for every token
    const void* F;           // element (a, f, j) at a * sa + f * sf + j * sj
    int64_t sa, sf, sj;
    int ld, rank, count;
    int dtype;               // 0 fp16, 1 bf16, 2 fp32
    int vec;                 // 16-bit type, j contiguous, every 8 values 16-byte aligned
};

__device__ __forceinline__ int lowrank_adapter(const LowRankEpi& e, int64_t m) {
    const int a = e.index ? __ldg(e.index + m) : 0;
    return (unsigned)a < (unsigned)e.count ? a : -1;
}

// A factor's value at element offset o.
__device__ __forceinline__ float factor_at(const void* F, int dtype, int64_t o) {
    switch (dtype) {
        case 0: return __half2float(__ldg(static_cast<const __half*>(F) + o));
        case 1: return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(F) + o));
        default: return __ldg(static_cast<const float*>(F) + o);
    }
}

__device__ __forceinline__ float2 pair16(uint32_t u, int dtype) {
    return dtype == 0 ? __half22float2(*reinterpret_cast<const __half2*>(&u))
                      : make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// 16 values j0 .. j0 + 15 of feature f of adapter a (0 beyond the rank).
__device__ __forceinline__ void lowrank_load16(const LowRankEpi& e, int a, int64_t f, int j0,
                                               float2 (&b)[8]) {
    const int64_t o = a * e.sa + f * e.sf;
    if (e.vec) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (j0 + 8 * h < e.rank)                     // (the rank is a multiple of 8)
                u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.F) + o + j0 + 8 * h));
            b[4 * h] = pair16(u.x, e.dtype);
            b[4 * h + 1] = pair16(u.y, e.dtype);
            b[4 * h + 2] = pair16(u.z, e.dtype);
            b[4 * h + 3] = pair16(u.w, e.dtype);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + 2 * i;
            b[i].x = j < e.rank ? factor_at(e.F, e.dtype, o + j * e.sj) : 0.0f;
            b[i].y = j + 1 < e.rank ? factor_at(e.F, e.dtype, o + (j + 1) * e.sj) : 0.0f;
        }
    }
}

// sum of 16 products with a token's T (16-byte aligned, the same for the warp).
__device__ __forceinline__ float lowrank_dot16(const float* t, const float2 (&b)[8]) {
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(t) + i);
        acc = __ffma2_rn(make_float2(q.x, q.y), b[2 * i], acc);
        acc = __ffma2_rn(make_float2(q.z, q.w), b[2 * i + 1], acc);
    }
    return __fadd_rn(acc.x, acc.y);
}

// The 16 factor values that a thread holds from one token to the next.
struct LowRankRegs {
    float2 b[8];
    int a, j0;
    __device__ __forceinline__ void init() { a = -1; j0 = 0; }
    __device__ __forceinline__ void want(const LowRankEpi& e, int adapter, int64_t f, int j) {
        if (adapter != a || j != j0) {
            lowrank_load16(e, adapter, f, j, b);
            a = adapter;
            j0 = j;
        }
    }
};

// v[i] += the term of token m + i (i < 8) at the thread's feature f.  Every
// lane of the warp has the same tokens.
__device__ __forceinline__ void lowrank_add8(const LowRankEpi& e, LowRankRegs& r, int64_t m,
                                             int64_t M, int64_t f, float (&v)[8]) {
    int a[8];
    bool same = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = m + i < M ? lowrank_adapter(e, m + i) : -1;
        same = same && a[i] == a[0];
    }
    if (same) {
        if (a[0] < 0) return;
        for (int j = 0; j < e.ld; j += 16) {
            r.want(e, a[0], f, j);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = __fadd_rn(v[i], lowrank_dot16(e.T + (m + i) * e.ld + j, r.b));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            if (m + i >= M) break;
            const int ai = lowrank_adapter(e, m + i);
            if (ai < 0) continue;
            float d = 0.0f;
            for (int j = 0; j < e.ld; j += 16) {
                r.want(e, ai, f, j);
                d = __fadd_rn(d, lowrank_dot16(e.T + (m + i) * e.ld + j, r.b));
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = k == i ? __fadd_rn(v[k], d) : v[k];
        }
    }
}

// The term of one (token, feature), for kernels whose lanes hold different
// tokens.
__device__ __forceinline__ float lowrank_term(const LowRankEpi& e, int64_t m, int64_t f) {
    const int a = lowrank_adapter(e, m);
    float d = 0.0f;
    if (a >= 0)
#pragma unroll 1
        for (int j = 0; j < e.ld; j += 16) {
            float2 b[8];
            lowrank_load16(e, a, f, j, b);
            d = __fadd_rn(d, lowrank_dot16(e.T + m * e.ld + j, b));
        }
    return d;
}

}  // namespace hqq
