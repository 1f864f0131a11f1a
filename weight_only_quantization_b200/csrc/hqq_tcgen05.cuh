// hqq_tcgen05.cuh -- what the tensor-memory kernels of the linear layer share:
// bounded mbarrier waits, TMA loads, tcgen05 descriptors, MMA, commit and
// tensor-memory reads, and the exact 3-bit decode of a pair of codes.
#pragma once
#include <cuda.h>

#include "hqq_unpack.cuh"

namespace hqq {

namespace {

constexpr uint64_t kWaitNs = 1000000000ull;   // 1 s per wait

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// One test of the phase; the waiting thread may be suspended in hardware for
// up to about 0.1 ms (the suspend-time hint) before the test fails, so that
// waiting warps take no issue slots from the warps doing work.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(100000)
        : "memory");
    return ok != 0;
}

// Bounded wait for the phase of `parity` to complete.  `abort` (shared) makes
// waits return false at once after any wait of the CTA has run out; `drain`
// waits ignore it (used to let the CTA's own copies and MMAs land).
__device__ __noinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* abort,
                                       int* status, bool drain) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try(bar, parity)) {
        if (!drain && *abort) return false;
        if (global_ns() - t0 > kWaitNs) {
            *abort = 1;
            if (status) atomicExch(status, 1);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// 2-D tiled TMA load (no multicast) of box {64 k, BN rows} at (k, row).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int k, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row), "r"(bar)
        : "memory");
}

// Shared-memory matrix descriptor of a K-major operand with the 128-byte
// swizzle: rows of 128 bytes, 8-row core-matrix groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4)   // start address / 16
           | ((uint64_t)1 << 16)                 // leading byte offset (unused with swizzle)
           | ((uint64_t)(1024 >> 4) << 32)       // stride byte offset: 1024 B
           | ((uint64_t)1 << 46)                 // descriptor version of sm_100
           | ((uint64_t)2 << 61);                // 128-byte swizzle
}

__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

__device__ __forceinline__ void fence_before_sync() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void fence_after_sync() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 8 consecutive fp32 columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&v)[8]) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Codes at bits b, b + 3 of x (b = 0, or 6 when B6) as exact floats: one
// logic operation per code, (x & mask) | magic with the mask as the immediate
// and the bits of 2^23 in a register (mg), then one fma pair.
// Constants of the 3-bit decode, made opaque once per thread so that they
// stay in registers (packed f32x2 operations take register pairs only):
// mg = the bits of 2^23, k20 = 2^20, k8 = 2^8, and per field pair (b, b + 3)
// with b = 0 or 6 the multipliers (2^-b, 2^-(b+3)) and offsets
// (-2^(23-b), -2^(20-b)) that turn 2^23 + c 2^b into c.
struct Dec3 {
    uint32_t mg, k20, k8;
    uint64_t i0, o0, i6, o6;                  // f32x2 pairs, low word first
    __device__ __forceinline__ void init() {
        mg = 0x4B000000u;
        k20 = 1u << 20;
        k8 = 1u << 8;
        auto pack = [](float lo, float hi) {
            return (uint64_t)__float_as_uint(lo) | ((uint64_t)__float_as_uint(hi) << 32);
        };
        i0 = pack(1.0f, 0.125f);
        o0 = pack(-8388608.0f, -1048576.0f);
        i6 = pack(0.015625f, 0.001953125f);
        o6 = pack(-131072.0f, -16384.0f);
        asm volatile("" : "+r"(mg), "+r"(k20), "+r"(k8));
        asm volatile("" : "+l"(i0), "+l"(o0), "+l"(i6), "+l"(o6));
    }
};

// fp16((c - z) s) of the codes at bits b, b + 3 of x (b = 0, or 6 when B6),
// packed in one word, as one block: the two fields into the mantissa of 2^23
// (one logic operation each), the exact codes (one f32x2 fma), fl32(c - z) and
// fl32(. s) (one f32x2 add and multiply, nz = (-z, -z), ss = (s, s)), the fp16
// pair.
template <int B6>
__device__ __forceinline__ uint32_t pair3_dq(uint32_t x, const Dec3& d, uint64_t nz, uint64_t ss) {
    constexpr uint32_t m0 = 7u << (B6 ? 6 : 0), m1 = m0 << 3;
    uint32_t h;
    asm("{\n\t.reg .b32 a, b, lo, hi;\n\t.reg .b64 ab, c;\n\t"
        "lop3.b32 a, %1, %2, %4, 0xEA;\n\t"
        "lop3.b32 b, %1, %3, %4, 0xEA;\n\t"
        "mov.b64 ab, {a, b};\n\t"
        "fma.rn.f32x2 c, ab, %5, %6;\n\t"
        "add.rn.f32x2 c, c, %7;\n\t"
        "mul.rn.f32x2 c, c, %8;\n\t"
        "mov.b64 {lo, hi}, c;\n\t"
        "cvt.rn.f16x2.f32 %0, hi, lo;\n\t}"
        : "=r"(h)
        : "r"(x), "n"(m0), "n"(m1), "r"(d.mg), "l"(B6 ? d.i6 : d.i0), "l"(B6 ? d.o6 : d.o0),
          "l"(nz), "l"(ss));
    return h;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn lookup_encode_fn() {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    EncodeTiledFn fn = nullptr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
        fn = reinterpret_cast<EncodeTiledFn>(p);
    cudaGetLastError();                               // a failed lookup leaves no error behind
    return fn;
}

// The driver's tensor-map encoder, looked up once (a function-local static is
// initialised exactly once even when several host threads call at once).
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = lookup_encode_fn();
    return fn;
}

}  // namespace

}  // namespace hqq
