// hqq_gemm.cuh -- the many-token products of a quantized matrix with a low-rank
// term (hqq_linear_adapters and its input gradient):
//
//   layer     Y[m, n]  = sum_k X[m, k]  W_hat[n, k] + sum_j T[m, j] B[n, j]
//   gradient  dX[m, k] = sum_n dY[m, n] W_hat[n, k] + sum_j P[m, j] A[j, k]
//
// with W_hat = fp16((code - z) s) formed inside the product and one rounding of
// the output.  Tensor cores: tcgen05.mma kind::f16, fp32 accumulators in tensor
// memory, the output transposed (features x tokens):
//   A = 128 features x 64 of the reduction, written to shared memory by 16
//       producer warps that unpack 64 codes a thread.  Layer: K-major.  Gradient
//       (TRANS): the same packed rows read as [64 n][128 k] and stored
//       k-contiguous (MN-major); the transposition is the MMA descriptor's.
//   B = bn tokens x 64 of the reduction by TMA.
// CG = 2 pairs two CTAs (cta_group::2): 256 features share one set of tokens of
// which each CTA stages half, so that X crosses from L2 once per pair and a stage
// of a 512-token tile takes 48 KiB instead of 80.  The pair's leader issues the
// MMAs; the peer's producers and its copies report to the leader's barriers.
// ks > 1 splits the reduction over a cluster; each CTA adds up and stores a
// share of the tile's tokens (partial sums travel through distributed shared
// memory, added in rank order).
// What the choice of bn, ks and CG weighs is at plan_gemm below.
//
// Warps: 0 TMA, 1 MMA and tensor memory, 2..17 producers, which also run the
// epilogue: the sums are read in the layout of an m16n8 MMA, the low-rank term is
// added to them 16 ranks a pass (factors in registers, T in shared memory) and the
// rounded outputs go through shared memory into rows of 64 bytes.  Tokens of several
// adapters in one block of eight are grouped by adapter first.  (On CUDA cores every
// product needs its own broadcast of T, four cycles of shared memory per 16 bytes:
// 28672 x 8192, 2048 tokens, rank 64: 1640 us against 1176.)
//
// What bounds it: at 512 tokens a tile 128 reduction steps take 0.97 us each where
// the MMAs need 0.74 (8192 x 8192 at 3 bits, 2048 tokens: 262 us, 1050 TFLOP/s); the
// rest is the pair's handshake and the producers' loads and decode (timing-only
// copies: 0.81 us without the code loads).  At up to 256 tokens a step takes 0.60 us
// whatever bn: producers and handshake.  What these were measured against: arrivals
// at cluster scope by every producer warp 1.66 us a step (they wait for the code
// loads in flight), waits as calls that read the clock 0.15 us more, 16 codes a
// thread instead of 64 1.05 us.  Every mbarrier wait is bounded (hqq_tcgen05.cuh); after one has
// run out the CTA still drains its own copies and MMAs, and the result is
// unspecified.
#pragma once
#include <cooperative_groups.h>

#include "hqq_lowrank_epi.cuh"
#include "hqq_tcgen05.cuh"

namespace hqq {

namespace cg = cooperative_groups;

namespace {

constexpr int kGmThreads = 576;
constexpr int kGmGroups = 4;                     // producer groups of four warps
constexpr int kGmM = 128;                        // features per CTA
constexpr int kGmK = 64;                         // reduction per stage
constexpr uint32_t kGmABytes = kGmM * kGmK * 2;
constexpr uint32_t kGmStageBytes = 196608;       // all stages together (192 KiB)
constexpr int kGmMaxStages = 8;
constexpr int kGmTries = 1000;                   // of a wait before it is timed (bounded)
constexpr int kGmOutRow = 40;                    // floats a staged token (banks apart)
constexpr int kGmWindow = 256;                   // tokens whose partial sums travel at once

struct GemmShape {
    int bn;                  // tokens per tile
    int nmma;                // tokens per MMA (bn, or bn / 2 above 256)
    int stages, ks;
    uint32_t b_bytes;        // staged tokens of a CTA: bn / CG rows of 128 bytes
    int vec;                 // 32 codes are one aligned run in memory (4 bits)
    int tile0;               // first feature tile of the launch
    int out_vec;             // the output's rows are whole aligned 16-byte runs
};

__device__ __forceinline__ bool mbar_try_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(100000)
        : "memory");
    return ok != 0;
}

// mbar_wait for a barrier that the other CTA of a pair reports to.
__device__ __noinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, volatile int* abort,
                                               int* status, bool drain) {
    if (mbar_try_cluster(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (!mbar_try_cluster(bar, parity)) {
        if (!drain && *abort) return false;
        if (global_ns() - t0 > kWaitNs) {
            *abort = 1;
            if (status) atomicExch(status, 1);
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Descriptor of an MN-major operand with the 128-byte swizzle: atoms of 8
// reduction rows x 64 values (128 bytes a row), the next 8 rows 1024 bytes on
// (stride offset), the next 64 values kGmHalf bytes on (leading offset).
constexpr uint32_t kGmHalf = 64 * 128;
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(kGmHalf >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

template <int CG>
__device__ __forceinline__ void gemm_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (CG == 1)
        mma_f16(d, a, b, idesc, accumulate);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Arrive on the barrier (of both CTAs of the pair) when the MMAs so far ended.
template <int CG>
__device__ __forceinline__ void gemm_commit(uint32_t bar, uint16_t pair) {
    if constexpr (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
            "h"(pair)
            : "memory");
}

// Read-only loads that stay where they are written (plain ones may be moved down
// to their use a step later).
__device__ __forceinline__ uint32_t ldnc(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldnc(const uint2* p) {
    uint2 v;
    asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ldnc(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t ldnc(const uint16_t* p) {
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ __half ldnc(const __half* p) {
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return __ushort_as_half(v);
}

// Eight fp32 columns of this warp's 32 tensor-memory lanes in the layout of two
// m16n8 MMA accumulators: v[h][e] = lane 16 h + lane / 4 + 8 (e / 2), column
// 2 (lane % 4) + e % 2.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[2][4]) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr));
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr + (16u << 16)));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i >> 2][i & 3] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const float (&v)[2][4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
        asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::
                         "r"(taddr + ((uint32_t)(16 * h) << 16)),
                     "r"(__float_as_uint(v[h][0])), "r"(__float_as_uint(v[h][1])),
                     "r"(__float_as_uint(v[h][2])), "r"(__float_as_uint(v[h][3]))
                     : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One fp32 column of this warp's 32 tensor-memory lanes; the caller waits for the
// load (tcgen05.wait::ld) before it uses the value.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return __uint_as_float(r);
}

__device__ __forceinline__ void tmem_wait8(float (&v)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]),
                   "+f"(v[7])
                 :
                 : "memory");
}

// 32 codes of one row from a multiple of 32, as loaded: nothing done with a
// loaded value here, which would wait for memory at once instead of at the
// group's next step.  A row ends after whole runs of 16, so the second half may be
// absent; absent codes decode to 0 (scale and zero 0).
template <int NBITS>
struct Codes32 {
    static constexpr int NW = NBITS == 3 ? 4 : NBITS;
    uint32_t w[NW];
    uint32_t off;                                // 3 bits: slot of code 0 in w[0]
    __half s[2], z[2];                           // of codes 0-15 and 16-31
};

// halves: 0, 1 or 2 of the runs present; vec: rows and buffer allow whole loads.
template <int NBITS, bool SMALL>
__device__ __forceinline__ void load32(const LinearParams& p, int64_t f, int halves, bool vec,
                                       Codes32<NBITS>& c) {
#pragma unroll
    for (int i = 0; i < Codes32<NBITS>::NW; ++i) c.w[i] = 0u;
    c.off = 0u;
    c.s[0] = c.s[1] = c.z[0] = c.z[1] = __float2half_rn(0.0f);
    if (halves == 0) return;
    if constexpr (NBITS == 3) {
        int64_t w0;
        if (SMALL) w0 = __umulhi(4u * (uint32_t)(f >> 3), 0xCCCCCCCDu) >> 2;    // f / 10
        else w0 = f / 10;
        c.off = (uint32_t)(f - 10 * w0);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed) + w0;
        const uint32_t slots = c.off + 16u * (uint32_t)halves;   // only words that hold them
        c.w[0] = ldnc(src);
        c.w[1] = ldnc(src + 1);
        if (slots > 20u) c.w[2] = ldnc(src + 2);
        if (slots > 30u) c.w[3] = ldnc(src + 3);
    } else if constexpr (NBITS == 8) {
        const uint2* src = reinterpret_cast<const uint2*>(p.packed + f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < 2 * halves) {
                const uint2 v = ldnc(src + i);
                c.w[2 * i] = v.x;
                c.w[2 * i + 1] = v.y;
            }
    } else if constexpr (NBITS == 4) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed) + (f >> 3);
        if (vec) {
            const uint4 v = ldnc(reinterpret_cast<const uint4*>(src));
            c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < 2 * halves) c.w[i] = ldnc(src + i);
        }
    } else if constexpr (NBITS == 2) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed) + (f >> 4);
        c.w[0] = ldnc(src);
        if (halves == 2) c.w[1] = ldnc(src + 1);
    } else {
        const uint16_t* src = reinterpret_cast<const uint16_t*>(p.packed) + (f >> 4);
        c.w[0] = ldnc(src);
        if (halves == 2) c.w[0] |= ldnc(src + 1) << 16;
    }
    const int64_t g = f >> p.log2_group;
    c.s[0] = p.sq.codes ? restore_meta_h(p.sq, g) : ldnc(p.scale + g);
    c.z[0] = p.zq.codes ? restore_meta_h(p.zq, g) : ldnc(p.zero + g);
    if (p.log2_group == 4 && halves == 2) {
        c.s[1] = p.sq.codes ? restore_meta_h(p.sq, g + 1) : ldnc(p.scale + g + 1);
        c.z[1] = p.zq.codes ? restore_meta_h(p.zq, g + 1) : ldnc(p.zero + g + 1);
    }
}

// Their fp16 weights, 8 per unit; one: both halves share the first scale and zero.
template <int NBITS>
__device__ __forceinline__ void decode32(const Codes32<NBITS>& c, bool one, const Dec3& d,
                                         uint4 (&o)[4]) {
    const float s0 = __half2float(c.s[0]), z0 = __half2float(c.z[0]);
    const float s1 = one ? s0 : __half2float(c.s[1]), z1 = one ? z0 : __half2float(c.z[1]);
    if constexpr (NBITS == 3) {
        // words re-based to codes 10 i .. 10 i + 9 in bits 0 ..; slots 0-3 from the
        // word, 4-7 from the word >> 12, 8-9 from the word >> 24 (multiply-highs)
        const uint32_t sh = 2u + 3u * c.off;
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = __funnelshift_r(c.w[i] << 2, i < 3 ? c.w[i < 3 ? i + 1 : 3] : 0u, sh);
        uint64_t ss[2], nz[2];
        asm("mov.b64 %0, {%1, %1};" : "=l"(ss[0]) : "f"(s0));
        asm("mov.b64 %0, {%1, %1};" : "=l"(nz[0]) : "f"(-z0));
        asm("mov.b64 %0, {%1, %1};" : "=l"(ss[1]) : "f"(s1));
        asm("mov.b64 %0, {%1, %1};" : "=l"(nz[1]) : "f"(-z1));
        uint32_t v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int sl = (2 * q) % 10, h = q >> 3;
            const uint32_t x = r[(2 * q) / 10];
            if (sl == 0) v[q] = pair3_dq<0>(x, d, nz[h], ss[h]);
            else if (sl == 2) v[q] = pair3_dq<1>(x, d, nz[h], ss[h]);
            else if (sl == 4) v[q] = pair3_dq<0>(__umulhi(x, d.k20), d, nz[h], ss[h]);
            else if (sl == 6) v[q] = pair3_dq<1>(__umulhi(x, d.k20), d, nz[h], ss[h]);
            else v[q] = pair3_dq<0>(__umulhi(x, d.k8), d, nz[h], ss[h]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) o[t] = make_uint4(v[4 * t], v[4 * t + 1], v[4 * t + 2], v[4 * t + 3]);
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const float s = t < 2 ? s0 : s1, z = t < 2 ? z0 : z1;
            if constexpr (NBITS == 8) o[t] = unit8_bytes(c.w[2 * t], c.w[2 * t + 1], z, s);
            else if constexpr (NBITS == 4) o[t] = unit8<4>(c.w[t], z, s);
            else if constexpr (NBITS == 2) o[t] = unit8<2>((c.w[t >> 1] >> (16 * (t & 1))) & 0xFFFFu, z, s);
            else o[t] = unit8<1>((c.w[0] >> (8 * t)) & 0xFFu, z, s);
        }
    }
}

// Grid: x = token tile * CG + CTA of the pair, y = feature tile (pair of tiles),
// z = part of the reduction; cluster (CG, 1, ks).
template <int NBITS, bool SMALL, bool TRANS, int CG>
__global__ void __launch_bounds__(kGmThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ LinearParams prm,
            const __grid_constant__ LowRankEpi lr, const __grid_constant__ GemmShape sh) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ uint64_t bars[3 * kGmMaxStages + 1];
    __shared__ uint32_t tmem_holder;
    __shared__ __align__(16) uint8_t stage_out[16][8 * kGmOutRow * 4];   // 8 tokens x 32 features a warp
    __shared__ int abort_flag;
    const int S = sh.stages, bn = sh.bn, parts = bn / sh.nmma;
    uint8_t* a_st = smem;
    uint8_t* b_st = smem + (uint32_t)S * kGmABytes;
    const uint32_t tmem_cols = bn <= 32 ? 32u : bn <= 64 ? 64u : bn <= 128 ? 128u : bn <= 256 ? 256u : 512u;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t c2 = CG == 2 ? blockIdx.x & 1u : 0u;            // CTA of the pair
    const int ks = sh.ks, zr = (int)blockIdx.z;
    const uint32_t leader = CG * (uint32_t)zr;                     // cluster rank
    const int64_t m0 = (int64_t)(blockIdx.x / CG) * bn;
    const int64_t n0 = (sh.tile0 + (int64_t)blockIdx.y * CG + c2) * kGmM;
    const int64_t features = TRANS ? prm.K : prm.N;
    const int KT = (int)(((TRANS ? prm.N : prm.K) + kGmK - 1) / kGmK);
    const int kt0 = (int)((int64_t)KT * zr / ks);
    const int nkt = (int)((int64_t)KT * (zr + 1) / ks) - kt0;
    const uint32_t bar0 = smem_u32(bars);
    auto full_a = [&](int s) { return bar0 + 8u * s; };
    auto full_b = [&](int s) { return bar0 + 8u * (kGmMaxStages + s); };
    auto empty = [&](int s) { return bar0 + 8u * (2 * kGmMaxStages + s); };
    const uint32_t done = bar0 + 8u * (3 * kGmMaxStages);
    volatile int* abrt = &abort_flag;
    auto wait = [&](uint32_t bar, uint32_t ph, bool drain) {
        // tries in line (each may be suspended in hardware): the call and its clock
        // reads cost a step's handshake 0.15 us
        for (int i = 0; i < kGmTries; ++i)
            if (mbar_try(bar, ph)) return;
        mbar_wait(bar, ph, abrt, prm.status, drain);
    };

    auto wait_cluster = [&](uint32_t bar, uint32_t ph) {
        for (int i = 0; i < kGmTries; ++i)
            if (mbar_try_cluster(bar, ph)) return;
        mbar_wait_cluster(bar, ph, abrt, prm.status, false);
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            // the producer group's warps, and on the leader the peer's whole stage
            mbar_init(full_a(s), 4 + (CG == 2 && c2 == 0 ? 1 : 0));
            mbar_init(full_b(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&xmap)) : "memory");
    }
    if (warp == 1) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_holder)), "r"(tmem_cols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(&tmem_holder)), "r"(tmem_cols) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    fence_before_sync();
    __syncthreads();
    if (CG == 2) cluster_sync_all();                     // the peer's barriers are ready
    fence_after_sync();
    const uint32_t tmem = tmem_holder;

    if (warp == 0) {
        if (lane == 0) {                                 // tokens by TMA
            const int rows = sh.nmma / CG;
            int s = 0;
            uint32_t ph = 0;
            for (int kt = 0; kt < nkt; ++kt) {
                wait(empty(s), ph ^ 1u, false);
                mbar_expect_tx(full_b(s), sh.b_bytes);
                for (int h = 0; h < parts; ++h)
                    tma_load_2d(smem_u32(b_st) + (uint32_t)s * sh.b_bytes + (uint32_t)(h * rows * 128),
                                &xmap, full_b(s), (kt0 + kt) * kGmK,
                                (int)m0 + h * sh.nmma + (int)c2 * rows);
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            // own loads landed, own stages read
            for (int kt = nkt > S ? nkt - S : 0; kt < nkt; ++kt) {
                wait(full_b(kt % S), (uint32_t)(kt / S) & 1u, true);
                wait(empty(kt % S), (uint32_t)(kt / S) & 1u, true);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && c2 == 0) {                      // MMA issue
            const uint32_t idesc = (1u << 4)             // D format: f32; A, B fp16
                                   | ((TRANS ? 1u : 0u) << 15)        // A is MN-major
                                   | ((uint32_t)(sh.nmma >> 3) << 17)
                                   | ((uint32_t)((kGmM * CG) >> 4) << 24);
            const uint16_t pair = (uint16_t)(3u << leader);
            const uint32_t half_b = (uint32_t)(sh.nmma / CG) * 128u;
            int s = 0;
            uint32_t ph = 0;
            for (int kt = 0; kt < nkt; ++kt) {
                wait(full_b(s), ph, false);
                if constexpr (CG == 1) wait(full_a(s), ph, false);
                else wait_cluster(full_a(s), ph);
                fence_after_sync();
                const uint32_t a0 = smem_u32(a_st) + (uint32_t)s * kGmABytes;
                const uint32_t b0 = smem_u32(b_st) + (uint32_t)s * sh.b_bytes;
                for (int h = 0; h < parts; ++h)
#pragma unroll
                    for (int k4 = 0; k4 < kGmK / 16; ++k4)
                        gemm_mma<CG>(tmem + (uint32_t)(h * sh.nmma),
                                     TRANS ? sw128_desc_mn(a0 + 2048u * k4) : sw128_desc(a0 + 32u * k4),
                                     sw128_desc(b0 + h * half_b + 32u * k4), idesc,
                                     (kt | k4) != 0 ? 1u : 0u);
                gemm_commit<CG>(empty(s), pair);         // stage free once these MMAs end
                if (++s == S) { s = 0; ph ^= 1u; }
            }
            gemm_commit<CG>(done, pair);
        } else if (CG == 2 && lane == 0) {
            // the peer's stage is whole: one report per stage, by a thread without
            // memory operations of its own (a producer's arrival at cluster scope would
            // wait for its code loads in flight)
            int s = 0;
            uint32_t ph = 0;
            for (int kt = 0; kt < nkt; ++kt) {
                wait(full_b(s), ph, false);
                wait(full_a(s), ph, false);
                mbar_arrive_cluster(map_to_rank(full_a(s), leader));
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
    } else {
        // ---- producers of W_hat: groups of four warps take the reduction steps in
        // turn, a thread two runs of 32 codes of its group's steps.  The runs are
        // decoded before the stage is free, the next step's codes are loaded (they
        // have the other groups' steps to arrive), then the weights are stored.  The
        // 8 lanes of a quarter-warp hold 8 rows of one column, so their 16-byte
        // stores hit the 8 distinct places of the swizzle.
        Dec3 dec;
        if constexpr (NBITS == 3) dec.init();
        const int group = (warp - 2) >> 2, w4 = (warp - 2) & 3;
        // run q: layer: row r + 64 q, codes 32 j .. (j < 2); TRANS: row r + 8 q,
        // codes 32 j .. (j < 4)
        const int r = 16 * w4 + (lane & 7) + (TRANS ? 0 : 8 * (lane >> 4));
        const int j = TRANS ? lane >> 3 : (lane >> 3) & 1;
        constexpr int kRunRows = TRANS ? 8 : 64;
        const int64_t row0 = (TRANS ? (int64_t)kt0 * kGmK : n0) + r;
        const int64_t col0 = (TRANS ? n0 : (int64_t)kt0 * kGmK) + 32 * j;
        const int64_t f0 = row0 * prm.K + col0;
        const bool one = prm.log2_group > 4, vec = sh.vec != 0;
        Codes32<NBITS> raw[2];
        auto fetch = [&](int kt) {
            const int64_t at = (int64_t)kt * kGmK, f = f0 + (TRANS ? at * prm.K : at);
            const int64_t left = prm.K - col0 - (TRANS ? 0 : at);
            const int halves = left >= 32 ? 2 : left > 0 ? 1 : 0;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                load32<NBITS, SMALL>(prm, f + (int64_t)(q * kRunRows) * prm.K,
                                     row0 + q * kRunRows + (TRANS ? at : 0) < prm.N ? halves : 0,
                                     vec, raw[q]);
        };
        // places of a run's 16-byte units in the tile
        uint32_t place[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            place[t] = (uint32_t)r * 128u + (TRANS ? (uint32_t)(j >> 1) * kGmHalf : 0u) +
                       ((uint32_t)((4 * (j & 1) + t) ^ (r & 7)) << 4);
        if (group < nkt) fetch(group);
        int s = group % S;
        uint32_t ph = 1u ^ ((uint32_t)(group / S) & 1u);
        for (int kt = group; kt < nkt; kt += kGmGroups) {
            uint4 o[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                // a lone first half: its scale must not decode the absent second one
                const bool whole = TRANS ? prm.K - col0 >= 32
                                         : prm.K - col0 - (int64_t)kt * kGmK >= 32;
                decode32<NBITS>(raw[q], one && whole, dec, o[q]);
            }
            if (kt + kGmGroups < nkt) fetch(kt + kGmGroups);
            wait(empty(s), ph, false);
            uint8_t* tile = a_st + (uint32_t)s * kGmABytes;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    *reinterpret_cast<uint4*>(tile + place[t] + (uint32_t)(q * kRunRows * 128)) = o[q][t];
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full_a(s));
            s += kGmGroups;
            while (s >= S) {
                s -= S;
                ph ^= 1u;
            }
        }
    }
    __syncwarp();
    wait(done, 0u, true);                                // every MMA of the tile ended
    fence_after_sync();
    __syncthreads();
    if (CG * ks > 1) cluster_sync_all();                 // ... in every CTA: stages are free

    // ---- epilogue: D[feature][token] -> Y[token][feature].  A warp reads the
    // tensor-memory lanes 32 (warp % 4) .. +31; the four producer warps of a
    // quarter share out the tokens, eight at a time.
    const bool epi = warp >= 2;
    const int grp = (warp - 2) >> 2;
    const int f = 32 * (warp & 3) + lane;                // feature within the tile
    const int64_t nf = n0 + f;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float* xbuf = reinterpret_cast<float*>(smem);        // the other parts' sums
    const int win = ks > 1 && bn > kGmWindow ? kGmWindow : bn;
    if (lr.T) wait_for_T();
    LowRankTile lt;
    lt.place(smem + (ks > 1 ? (uint32_t)win * kGmM * 4u : 0u),
             (uint32_t)S * (kGmABytes + sh.b_bytes) - (ks > 1 ? (uint32_t)win * kGmM * 4u : 0u));
    for (int w0 = 0; w0 < bn; w0 += win) {
        const int width = bn - w0 < win ? bn - w0 : win;
        const int share = width / ks, c0 = w0 + zr * share;        // this CTA's tokens
        if (ks > 1) {
            if (w0) cluster_sync_all();                  // the last window has been added up
            if (epi)
                for (int q = 1; q < ks; ++q) {
                    const int to = (zr + q) % ks, slot = zr < to ? zr : zr - 1;
                    const uint32_t dst =
                        map_to_rank(smem_u32(xbuf), CG * (uint32_t)to + c2) +
                        (uint32_t)(slot * share * kGmM + f) * 4u;
#pragma unroll 1
                    for (int c = 8 * grp; c < share; c += 32) {
                        float v[8];
                        tmem_ld8(trow + (uint32_t)(w0 + to * share + c), v);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(
                                             dst + (uint32_t)((c + i) * kGmM) * 4u),
                                         "f"(v[i])
                                         : "memory");
                    }
                }
        }
        if (lr.T) lt.stage(lr, m0 + c0, share, prm.M, threadIdx.x, kGmThreads);
        if (ks > 1) cluster_sync_all();
        else __syncthreads();
        // blocks that mix adapters (or whose T is not staged): tokens in groups
        const bool mixed = lr.T && __syncthreads_or((int)threadIdx.x < share && lt.mark(threadIdx.x));
        if (mixed) {
            lt.group(share, threadIdx.x, kGmThreads);
            __syncthreads();
        }
        if (epi) {
            // eight tokens at a time in the layout of an m16n8 MMA, stored through a
            // transposition in shared memory: 64 bytes of a token's row for 4 lanes
            LowRankFrag frag;
            frag.init();
            uint8_t* out = stage_out[warp - 2];
            const uint32_t out_row = smem_u32(out) + (uint32_t)((lane & 7) * 64 + (lane >> 3) * 16);
            float* outf = reinterpret_cast<float*>(out);
            const int64_t fb = n0 + 32 * (warp & 3);     // the warp's features
            // (16 ranks a pass: the factor's values stay in registers, the sums go back
            // to tensor memory between passes)
            const int ranks = lr.T ? lr.ld : 16;
#pragma unroll 1
            for (int j = 0; j < ranks; j += 16)
#pragma unroll 1
            for (int c = 8 * grp; c < share; c += 32) {
                if (mixed && lt.key[c] != LowRankTile::kFast) continue;   // (below)
                float v[2][4];
                tmem_ld_frag(trow + (uint32_t)(c0 + c), v);
                if (lr.T && lt.adapter[c] >= 0)
                    lt.add_block(lr, frag, lt.adapter[c], c + (lane >> 2), j, fb, features, lane, v);
                if (j + 16 < ranks) {
                    tmem_st_frag(trow + (uint32_t)(c0 + c), v);
                    continue;
                }
                for (int q = 0; q < ks - 1; ++q) {
                    const float* src = xbuf + ((size_t)q * share + c + 2 * (lane & 3)) * kGmM +
                                       32 * (warp & 3) + (lane >> 2);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            v[h][i] = __fadd_rn(v[h][i], src[(i & 1) * kGmM + 16 * h + 8 * (i >> 1)]);
                }
                uint32_t w[4];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const __half2 p = __floats2half2_rn(v[h][2 * i], v[h][2 * i + 1]);
                        w[2 * h + i] = *reinterpret_cast<const uint32_t*>(&p);
                    }
                __syncwarp();                            // the last eight have been read
                asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::
                                 "r"(out_row), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
                __syncwarp();
                const uint4 u = *reinterpret_cast<const uint4*>(out + 16 * lane);
                const int64_t m = m0 + c0 + c + (lane >> 2), fo = fb + 8 * (lane & 3);
                if (m < prm.M) {
                    __half* dst = prm.Y + m * features + fo;
                    if (sh.out_vec && fo < features) {
                        *reinterpret_cast<uint4*>(dst) = u;
                    } else {
                        const __half* hs = reinterpret_cast<const __half*>(&u);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (fo + i < features) dst[i] = hs[i];
                    }
                }
            }
            // groups of up to eight tokens with one adapter: their columns go through
            // shared memory to the MMA's layout and back, so that an adapter's factor
            // is loaded once a group and not once a token
            if (mixed)
#pragma unroll 1
                for (int q = grp; q < *lt.ngroups; q += 4) {
                    const int first = lt.groups[q] & 0xffff, len = lt.groups[q] >> 16;
                    const int a = lt.adapter[lt.sorted[first]];
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = tmem_ld1(trow + (uint32_t)(c0 + lt.sorted[first + (i < len ? i : 0)]));
                    tmem_wait8(v);
                    if (a >= 0) {
                        __syncwarp();                    // the last group has been read
#pragma unroll
                        for (int i = 0; i < 8; ++i) outf[i * kGmOutRow + lane] = v[i];
                        __syncwarp();
                        float w[2][4];
                        float* at = outf + 2 * (lane & 3) * kGmOutRow + (lane >> 2);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[h][i] = at[(i & 1) * kGmOutRow + 16 * h + 8 * (i >> 1)];
                        const int tok = (lane >> 2) < len ? lt.sorted[first + (lane >> 2)] : -1;
                        for (int j = 0; j < lr.ld; j += 32) {    // (two loads in flight)
                            LowRankFrag other;
                            if (frag.a != a || frag.j != j) frag.load(lr, a, fb, features, j, lane);
                            if (j + 16 < lr.ld) other.load(lr, a, fb, features, j + 16, lane);
                            lt.add_block(lr, frag, a, tok, j, fb, features, lane, w);
                            if (j + 16 < lr.ld)
                                lt.add_block(lr, other, a, tok, j + 16, fb, features, lane, w);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int i = 0; i < 4; ++i) at[(i & 1) * kGmOutRow + 16 * h + 8 * (i >> 1)] = w[h][i];
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] = outf[i * kGmOutRow + lane];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (i >= len) break;
                        const int c = lt.sorted[first + i];
                        for (int r = 0; r < ks - 1; ++r)
                            v[i] = __fadd_rn(v[i], xbuf[((size_t)r * share + c) * kGmM + f]);
                        const int64_t m = m0 + c0 + c;
                        if (m < prm.M && nf < features) prm.Y[m * features + nf] = __float2half_rn(v[i]);
                    }
                }
        }
        __syncwarp();
    }
    fence_before_sync();
    __syncthreads();
    if (CG * ks > 1) cluster_sync_all();                 // no CTA leaves before its peers
    if (warp == 1) {
        fence_after_sync();
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(tmem_cols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                         "r"(tmem_cols) : "memory");
    }
}

struct GemmPlan {
    int cg, ks, bn;
    int64_t rows;            // rows of feature tiles (cg tiles each) that fill whole rounds
    double cost, round;      // us: all of it, one round
};

// Tile choice, from the times of every (CG, ks, bn) on four matrices and 64 to
// 2048 tokens: a round of tiles takes its reduction steps plus a fixed part,
//   CG = 1   0.60 us a step whatever bn (producers and handshakes),
//   CG = 2   max(0.74, 0.0019 bn) us a step (the handshake between the CTAs; from
//            384 tokens the MMAs),
// e.g. 4096 x 4096 at 4 bits (64 steps): 256 tokens 47 us as one CTA, 32 split by 2
// and 23 split by 4; 2048 tokens 96 us in tiles of 256 and 73 in pairs of 512.  A
// round holds one CTA per SM, fewer where clusters leave part of a GPC's SMs
// over: four-CTA clusters reach 16 SMs of 18, and of eight CTAs only a few run at
// once (splits by 8 measured slower wherever more than 8 clusters were needed).
GemmPlan plan_gemm(int64_t M, int64_t features, int64_t depth, int sms) {
    const int64_t steps = (depth + kGmK - 1) / kGmK, tiles = (features + kGmM - 1) / kGmM;
    GemmPlan best = {1, 1, 16, 0, 1e30, 0.0};
    for (int cg = 1; cg <= 2; ++cg)
        for (int ks = 1; ks * cg <= 8; ks *= 2) {
            if (ks > 1 && steps < 4 * ks) break;
            const int size = cg * ks;
            const int64_t slots = size == 1 ? sms : size == 2 ? sms / 2 * 2
                                  : size == 4 ? sms * 16 / 18 / 4 * 4 : 64;
            // bn: every MMA a multiple of 16 tokens a CTA (above 256 two MMAs), every
            // share of a split a multiple of 8
            const int unit = 8 * ks > 16 * cg ? 8 * ks : 16 * cg, most = 256 * cg;
            const int64_t whole = (M + unit - 1) / unit * unit;
            int bn = whole < most ? (int)whole : most;
            if (bn > 256) bn = (bn + 63) / 64 * 64;
            for (; bn > 0; bn -= bn > 256 ? 64 : unit > 32 ? unit : 32) {
                const int64_t ctas = (M + bn - 1) / bn * ((tiles + cg - 1) / cg) * size;
                if (size == 8 && ctas > slots) break;
                const double rounds = (double)((ctas + slots - 1) / slots);
                const double step = cg == 1 ? 0.60 : 0.0019 * bn > 0.74 ? 0.0019 * bn : 0.74;
                const double one = (double)((steps + ks - 1) / ks) * step +
                                   (cg == 1 ? 8.5 : 13.0) + (ks > 1 ? 0.02 : 0.01) * bn;
                if (rounds * one < best.cost)
                    best = {cg, ks, bn, (ctas / slots) * slots / ((M + bn - 1) / bn * size),
                            rounds * one, one};
                if (bn <= 64 || bn % unit != 0) break;
            }
        }
    return best;
}

// Feature tiles tile0 .. tile0 + tiles - 1 (kGmM features each) of the output.
template <int NBITS, bool SMALL, bool TRANS, int CG>
cudaError_t launch_gemm_cg(const LinearParams& prm, const LowRankEpi& lr, const void* X, int64_t ld,
                           const GemmPlan& plan, int64_t tile0, int64_t tiles, bool beside_T,
                           cudaStream_t stream) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const int64_t depth = TRANS ? prm.N : prm.K;
    GemmShape sh;
    sh.tile0 = (int)tile0;
    sh.out_vec = (TRANS ? prm.K : prm.N) % 8 == 0 && (reinterpret_cast<uintptr_t>(prm.Y) & 15u) == 0;
    sh.bn = plan.bn;
    sh.nmma = plan.bn > 256 ? plan.bn / 2 : plan.bn;
    sh.ks = plan.ks;
    sh.vec = prm.K % 32 == 0 && (reinterpret_cast<uintptr_t>(prm.packed) & 15u) == 0;
    sh.b_bytes = (uint32_t)(plan.bn / CG) * 128u;
    const uint32_t fit = kGmStageBytes / (kGmABytes + sh.b_bytes);
    sh.stages = (int)(fit < (uint32_t)kGmMaxStages ? fit : (uint32_t)kGmMaxStages);
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)depth, (cuuint64_t)prm.M};
    const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    const cuuint32_t box[2] = {(cuuint32_t)kGmK, (cuuint32_t)(sh.nmma / CG)};
    const cuuint32_t estr[2] = {1, 1};
    if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(X), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    auto kern = gemm_kernel<NBITS, SMALL, TRANS, CG>;
    // stages (also the epilogue's windows of partial sums and T) and alignment
    const size_t smem = 1024 + kGmStageBytes;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)plan.ks;
    cfg.gridDim = dim3((unsigned)((prm.M + plan.bn - 1) / plan.bn * CG),
                       (unsigned)((tiles + CG - 1) / CG), (unsigned)plan.ks);
    cfg.blockDim = dim3(kGmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside_T ? 2 : 1;          // beside the kernel that writes T
    return cudaLaunchKernelEx(&cfg, kern, map, prm, lr, sh);
}

template <int NBITS, bool SMALL, bool TRANS>
cudaError_t launch_gemm_n(const LinearParams& prm, const LowRankEpi& lr, const void* X, int64_t ld,
                          cudaStream_t stream) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t features = TRANS ? prm.K : prm.N, depth = TRANS ? prm.N : prm.K;
    const int64_t tiles = (features + kGmM - 1) / kGmM;
    auto launch = [&](const GemmPlan& plan, int64_t tile0, int64_t count, bool beside_T) {
        return plan.cg == 2
            ? launch_gemm_cg<NBITS, SMALL, TRANS, 2>(prm, lr, X, ld, plan, tile0, count, beside_T, stream)
            : launch_gemm_cg<NBITS, SMALL, TRANS, 1>(prm, lr, X, ld, plan, tile0, count, beside_T, stream);
    };
    const GemmPlan plan = plan_gemm(prm.M, features, depth, sms);
    // A nearly empty last round is a launch of its own, with the tiles that suit
    // what is left: the gate matrix at 2048 tokens is 448 pair tiles, 6 rounds of 74
    // and 4 tiles over (a seventh round of 142 us; on their own about 40).
    const int64_t whole = plan.rows * plan.cg;
    if (whole > 0 && whole < tiles) {
        const GemmPlan rest = plan_gemm(prm.M, features - whole * kGmM, depth, sms);
        const int64_t per_row = (prm.M + plan.bn - 1) / plan.bn * plan.cg * plan.ks;
        const int64_t size = plan.cg * plan.ks;
        const int64_t slots = size == 4 ? sms * 16 / 18 / 4 * 4 : size == 2 ? sms / 2 * 2 : size == 1 ? sms : 64;
        const double first = (double)((plan.rows * per_row + slots - 1) / slots) * plan.round;
        if (first + rest.cost + 3.0 < plan.cost) {
            const cudaError_t e = launch(plan, 0, whole, lr.T != nullptr);
            return e == cudaSuccess ? launch(rest, whole, tiles - whole, false) : e;
        }
    }
    return launch(plan, 0, tiles, lr.T != nullptr);
}

// X: [M, K] (TRANS: dY, [M, N]), rows ld values apart, 16-byte aligned.
template <bool TRANS>
cudaError_t launch_gemm(const LinearParams& prm, const LowRankEpi& lr, const void* X, int64_t ld,
                        int nbits, cudaStream_t stream) {
    const bool small = prm.N * prm.K / 8 < ((int64_t)1 << 30);
    switch (nbits) {
        case 1: return launch_gemm_n<1, true, TRANS>(prm, lr, X, ld, stream);
        case 2: return launch_gemm_n<2, true, TRANS>(prm, lr, X, ld, stream);
        case 4: return launch_gemm_n<4, true, TRANS>(prm, lr, X, ld, stream);
        case 8: return launch_gemm_n<8, true, TRANS>(prm, lr, X, ld, stream);
        case 3:
            return small ? launch_gemm_n<3, true, TRANS>(prm, lr, X, ld, stream)
                         : launch_gemm_n<3, false, TRANS>(prm, lr, X, ld, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

}  // namespace hqq
