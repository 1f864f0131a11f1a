// hqq_tf32.cuh -- what the adapters' kernels share: fp32 values as two tf32 halves,
// the warp-level tf32 MMA, and a factor's value of any type.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace hqq {

// x = hi + lo as tf32 operands of an MMA, which reads a value's upper 19 bits: hi is
// x rounded to nearest by an integer addition (the conversion instruction measured
// slower), lo the exact difference of at most 12 bits, whose last one may be cut off, so
// that the rest is at most 2^-23 |x|.  hi is kept finite (the minimum of the absolute
// values, with x's sign, is the bound for a NaN): the NaN of the GPU's arithmetic has
// every bit but the sign set, and the addition would carry it to -0, values above the
// bound to infinity.  A NaN or an infinity is in lo instead.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
    constexpr float kMax = 0x1.ffcp127f;                 // the largest finite tf32 value
    float y;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(kMax));
    hi = (__float_as_uint(y) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(__fsub_rn(x, __uint_as_float(hi)));
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A factor's value at element offset o; dtype 0 fp16, 1 bf16, 2 fp32.
__device__ __forceinline__ float factor_at(const void* F, int dtype, int64_t o) {
    switch (dtype) {
        case 0: return __half2float(__ldg(static_cast<const __half*>(F) + o));
        case 1: return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(F) + o));
        default: return __ldg(static_cast<const float*>(F) + o);
    }
}

}  // namespace hqq
