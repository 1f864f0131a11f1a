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
//       producer warps that unpack 16 codes a thread.  Layer: K-major.  Gradient
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
// Warps: 0 TMA, 1 MMA and tensor memory, 2..17 producers; all join the epilogue,
// where the low-rank term is added in fp32 from factors in registers and T in
// shared memory.  Every mbarrier wait is bounded (hqq_tcgen05.cuh); after one has
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
constexpr int kGmProducers = 16;                 // warps
constexpr int kGmM = 128;                        // features per CTA
constexpr int kGmK = 64;                         // reduction per stage
constexpr uint32_t kGmABytes = kGmM * kGmK * 2;
constexpr uint32_t kGmStageBytes = 196608;       // all stages together (192 KiB)
constexpr int kGmMaxStages = 8;
constexpr int kGmWindow = 256;                   // tokens whose partial sums travel at once
constexpr int kGmAhead = 4;                      // reduction steps of codes in registers

struct GemmShape {
    int bn;                  // tokens per tile
    int nmma;                // tokens per MMA (bn, or bn / 2 above 256)
    int stages, ks;
    uint32_t b_bytes;        // staged tokens of a CTA: bn / CG rows of 128 bytes
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

// 16 consecutive codes of one row (inside one group; rows are whole runs of 16)
// as loaded, with their (scale, zero).  Absent ones decode to 0.
template <int NBITS>
struct Codes16 {
    static constexpr int NW = NBITS == 8 ? 4 : NBITS == 4 ? 2 : NBITS == 3 ? 3 : 1;
    uint32_t w[NW];
    uint32_t off;                                // 3 bits: slot of code 0 in w[0]
    __half2 sz;
};

template <int NBITS, bool SMALL>
__device__ __forceinline__ void load16(const LinearParams& p, int64_t f, bool ok,
                                       Codes16<NBITS>& c) {
#pragma unroll
    for (int i = 0; i < Codes16<NBITS>::NW; ++i) c.w[i] = 0u;
    c.off = 0u;
    c.sz = __float2half2_rn(0.0f);
    if (!ok) return;
    if constexpr (NBITS == 3) {
        int64_t w0;
        if (SMALL) w0 = __umulhi(4u * (uint32_t)(f >> 3), 0xCCCCCCCDu) >> 2;    // f / 10
        else w0 = f / 10;
        c.off = (uint32_t)(f - 10 * w0);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed) + w0;
        c.w[0] = __ldg(src);
        c.w[1] = __ldg(src + 1);
        if (c.off > 4u) c.w[2] = __ldg(src + 2);     // only words that hold its codes
    } else if constexpr (NBITS == 8) {
        const uint2* src = reinterpret_cast<const uint2*>(p.packed + f);
        const uint2 a = __ldg(src), b = __ldg(src + 1);
        c.w[0] = a.x; c.w[1] = a.y; c.w[2] = b.x; c.w[3] = b.y;
    } else if constexpr (NBITS == 4) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.packed) + (f >> 3);
        c.w[0] = __ldg(src);
        c.w[1] = __ldg(src + 1);
    } else if constexpr (NBITS == 2) {
        c.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p.packed) + (f >> 4));
    } else {
        c.w[0] = __ldg(reinterpret_cast<const uint16_t*>(p.packed) + (f >> 4));
    }
    c.sz = group_sz(p, f >> p.log2_group);
}

// Their fp16 weights: codes 0 .. 7 and 8 .. 15.
template <int NBITS>
__device__ __forceinline__ void decode16(const Codes16<NBITS>& c, const Dec3& d, uint4 (&o)[2]) {
    const float s = __low2float(c.sz), z = __high2float(c.sz);
    if constexpr (NBITS == 3) {
        // words re-based to codes 0 .. 9 and 10 .. 15 in bits 0 ..
        const uint32_t sh = 2u + 3u * c.off;
        const uint32_t r0 = __funnelshift_r(c.w[0] << 2, c.w[1], sh);
        const uint32_t r1 = __funnelshift_r(c.w[1] << 2, c.w[2], sh);
        uint64_t ss, nz;
        asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
        asm("mov.b64 %0, {%1, %1};" : "=l"(nz) : "f"(-z));
        const uint32_t r0h = __umulhi(r0, d.k20);                 // >> 12
        o[0].x = pair3_dq<0>(r0, d, nz, ss);
        o[0].y = pair3_dq<1>(r0, d, nz, ss);
        o[0].z = pair3_dq<0>(r0h, d, nz, ss);
        o[0].w = pair3_dq<1>(r0h, d, nz, ss);
        o[1].x = pair3_dq<0>(__umulhi(r0, d.k8), d, nz, ss);      // >> 24
        o[1].y = pair3_dq<0>(r1, d, nz, ss);
        o[1].z = pair3_dq<1>(r1, d, nz, ss);
        o[1].w = pair3_dq<0>(__umulhi(r1, d.k20), d, nz, ss);
    } else if constexpr (NBITS == 8) {
        o[0] = unit8_bytes(c.w[0], c.w[1], z, s);
        o[1] = unit8_bytes(c.w[2], c.w[3], z, s);
    } else if constexpr (NBITS == 4) {
        o[0] = unit8<4>(c.w[0], z, s);
        o[1] = unit8<4>(c.w[1], z, s);
    } else if constexpr (NBITS == 2) {
        o[0] = unit8<2>(c.w[0] & 0xFFFFu, z, s);
        o[1] = unit8<2>(c.w[0] >> 16, z, s);
    } else {
        o[0] = unit8<1>(c.w[0] & 0xFFu, z, s);
        o[1] = unit8<1>(c.w[0] >> 8, z, s);
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
    const int64_t n0 = ((int64_t)blockIdx.y * CG + c2) * kGmM;
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
        if constexpr (CG == 1) mbar_wait(bar, ph, abrt, prm.status, drain);
        else mbar_wait_cluster(bar, ph, abrt, prm.status, drain);
    };

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            // producer warps of both CTAs, and the peer's staged tokens
            mbar_init(full_a(s), CG == 1 ? kGmProducers : 2 * kGmProducers + 1);
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
                wait(full_a(s), ph, false);
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
        } else if (CG == 2 && lane == 0) {               // the peer's tokens are staged
            int s = 0;
            uint32_t ph = 0;
            for (int kt = 0; kt < nkt; ++kt) {
                wait(full_b(s), ph, false);
                mbar_arrive_cluster(map_to_rank(full_a(s), leader));
                if (++s == S) { s = 0; ph ^= 1u; }
            }
        }
    } else {
        // ---- producers of W_hat: 16 codes a thread and step; the 8 lanes of a
        // quarter-warp hold 8 rows of one column, so their 16-byte stores hit the
        // 8 distinct places of the swizzle
        Dec3 dec;
        if constexpr (NBITS == 3) dec.init();
        const int pw = warp - 2;
        const int r = TRANS ? (pw & 7) * 8 + (lane & 7) : pw * 8 + (lane & 7);
        const int j = TRANS ? (pw >> 3) * 4 + (lane >> 3) : lane >> 3;     // 16 codes from 16 j
        const int64_t row0 = TRANS ? (int64_t)kt0 * kGmK + r : n0 + r;
        const int64_t col0 = TRANS ? n0 + 16 * j : (int64_t)kt0 * kGmK + 16 * j;
        auto fetch = [&](int kt, Codes16<NBITS>& c) {
            const int64_t row = TRANS ? row0 + (int64_t)kt * kGmK : row0;
            const int64_t col = TRANS ? col0 : col0 + (int64_t)kt * kGmK;
            load16<NBITS, SMALL>(prm, row * prm.K + col, row < prm.N && col < prm.K, c);
        };
        // places of the thread's two 16-byte units in the tile
        const uint32_t base = (uint32_t)r * 128u + (TRANS ? (uint32_t)(j >> 2) * kGmHalf : 0u);
        const uint32_t u0 = base + ((uint32_t)(((2 * j) & 7) ^ (r & 7)) << 4);
        const uint32_t u1 = base + ((uint32_t)(((2 * j + 1) & 7) ^ (r & 7)) << 4);
        Codes16<NBITS> ring[kGmAhead];
#pragma unroll
        for (int u = 0; u < kGmAhead - 1; ++u)
            if (u < nkt) fetch(u, ring[u]);
        int s = 0;
        uint32_t ph = 1;
        for (int kb = 0; kb < nkt; kb += kGmAhead) {
#pragma unroll
            for (int u = 0; u < kGmAhead; ++u) {
                const int kt = kb + u;
                if (kt < nkt) {
                    if (kt + kGmAhead - 1 < nkt)
                        fetch(kt + kGmAhead - 1, ring[(u + kGmAhead - 1) % kGmAhead]);
                    uint4 o[2];
                    decode16<NBITS>(ring[u], dec, o);
                    wait(empty(s), ph, false);
                    uint8_t* tile = a_st + (uint32_t)s * kGmABytes;
                    *reinterpret_cast<uint4*>(tile + u0) = o[0];
                    *reinterpret_cast<uint4*>(tile + u1) = o[1];
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (CG == 1) mbar_arrive(full_a(s));
                        else mbar_arrive_cluster(map_to_rank(full_a(s), leader));
                    }
                    if (++s == S) { s = 0; ph ^= 1u; }
                }
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
    const int64_t nf = n0 + f, nfc = nf < features ? nf : features - 1;
    const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float* xbuf = reinterpret_cast<float*>(smem);        // the other parts' sums
    const int win = ks > 1 && bn > kGmWindow ? kGmWindow : bn;
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
        if (epi) {
            LowRankRegs32 regs;
            regs.init();
#pragma unroll 1
            for (int c = 8 * grp; c < share; c += 32) {
                float v[8];
                tmem_ld8(trow + (uint32_t)(c0 + c), v);
                for (int q = 0; q < ks - 1; ++q) {
                    const float* src = xbuf + (size_t)q * share * kGmM + f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(v[i], src[(c + i) * kGmM]);
                }
                if (lr.T) lt.add8(lr, regs, c, nfc, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t m = m0 + c0 + c + i;
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
};

// Tile choice.  A reduction step of a CTA takes about max(kStep, kToken bn) us
// (decoding 128 x 64 weights, or the MMAs of bn tokens), a tile kTile us besides
// its steps and a split kSplit more; the tiles run in rounds of one CTA per SM.
GemmPlan plan_gemm(int64_t M, int64_t features, int64_t depth, int sms) {
    constexpr double kStep = 0.50, kToken = 0.00155, kTile = 5.0, kSplit = 3.0;
    const int64_t steps = (depth + kGmK - 1) / kGmK, tiles = (features + kGmM - 1) / kGmM;
    GemmPlan best = {1, 1, 16};
    double cost = 1e30;
    for (int cg = 1; cg <= 2; ++cg)
        for (int ks = 1; ks * cg <= 8; ks *= 2) {
            if (ks > 1 && steps < 4 * ks) break;
            // bn: every MMA a multiple of 16 tokens a CTA (above 256 two MMAs), every
            // share of a split a multiple of 8
            const int unit = 8 * ks > 16 * cg ? 8 * ks : 16 * cg, most = 256 * cg;
            const int64_t whole = (M + unit - 1) / unit * unit;
            int bn = whole < most ? (int)whole : most;
            if (bn > 256) bn = (bn + 63) / 64 * 64;
            for (; bn > 0; bn -= bn > 256 ? 64 : unit > 32 ? unit : 32) {
                const int64_t ctas = (M + bn - 1) / bn * ((tiles + cg - 1) / cg) * cg * ks;
                const int64_t slots = sms / cg * cg;
                const double rounds = (double)((ctas + slots - 1) / slots);
                const double step = kStep > kToken * bn ? kStep : kToken * bn;
                const double c = rounds * ((double)((steps + ks - 1) / ks) * step + kTile +
                                           (ks > 1 ? kSplit : 0.0) + 0.004 * bn / ks);
                if (c < cost) {
                    cost = c;
                    best = {cg, ks, bn};
                }
                if (bn <= 64 || bn % unit != 0) break;
            }
        }
    return best;
}

template <int NBITS, bool SMALL, bool TRANS, int CG>
cudaError_t launch_gemm_cg(const LinearParams& prm, const LowRankEpi& lr, const void* X, int64_t ld,
                           const GemmPlan& plan, cudaStream_t stream) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    const int64_t depth = TRANS ? prm.N : prm.K, features = TRANS ? prm.K : prm.N;
    GemmShape sh;
    sh.bn = plan.bn;
    sh.nmma = plan.bn > 256 ? plan.bn / 2 : plan.bn;
    sh.ks = plan.ks;
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
    const int64_t tiles = (features + kGmM - 1) / kGmM;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = (unsigned)plan.ks;
    cfg.gridDim = dim3((unsigned)((prm.M + plan.bn - 1) / plan.bn * CG),
                       (unsigned)((tiles + CG - 1) / CG), (unsigned)plan.ks);
    cfg.blockDim = dim3(kGmThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, map, prm, lr, sh);
}

template <int NBITS, bool SMALL, bool TRANS>
cudaError_t launch_gemm_n(const LinearParams& prm, const LowRankEpi& lr, const void* X, int64_t ld,
                          cudaStream_t stream) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const GemmPlan plan = plan_gemm(prm.M, TRANS ? prm.K : prm.N, TRANS ? prm.N : prm.K, sms);
    return plan.cg == 2 ? launch_gemm_cg<NBITS, SMALL, TRANS, 2>(prm, lr, X, ld, plan, stream)
                        : launch_gemm_cg<NBITS, SMALL, TRANS, 1>(prm, lr, X, ld, plan, stream);
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
