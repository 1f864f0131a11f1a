// hqq_lowrank_epi.cuh -- the low-rank term that the linear-layer kernels add to
// their fp32 sums: for token m with adapter a and output feature f
//   sum_j T[m, j] * F[a, f, j],
// T [M, ld] fp32 already scaled (hqq_adapters.cu), ld = the rank rounded up to 16
// with zeros behind it; F is the adapters' second factor (B for the layer, A for
// its input gradient) in fp16, bf16 or fp32, addressed by strides.  The few-token
// kernels sum over j in fp32 fused multiply-adds, the tensor-memory kernel in tf32
// MMAs with T (and fp32 factors) split into two halves.  A token without an adapter
// has no term (its row of T may hold anything).
#pragma once
#include "hqq_params.cuh"
#include "hqq_tf32.cuh"

namespace hqq {

// The kernel that adds the term starts before the one that writes T has ended
// (programmatic dependent launch): it waits here before its first read of T, and
// reads T from L2, where that kernel's writes are.
__device__ __forceinline__ void wait_for_T() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
        const float4 q = __ldcg(reinterpret_cast<const float4*>(t) + i);
        acc = __ffma2_rn(make_float2(q.x, q.y), b[2 * i], acc);
        acc = __ffma2_rn(make_float2(q.z, q.w), b[2 * i + 1], acc);
    }
    return __fadd_rn(acc.x, acc.y);
}

// 16 ranks (from j) of an adapter's factor at a warp's 32 features as MMA operands:
// x[h][r][i] = feature 16 h + 8 r + lane / 4, rank j + 4 (lane % 4) + i (the MMA's
// reduction index is permuted alike in both operands, so that a lane's four ranks
// are adjacent).
struct LowRankFrag {
    float x[2][2][4];
    int a, j;
    __device__ __forceinline__ void init() { a = -1; j = 0; }
    __device__ __forceinline__ void load(const LowRankEpi& e, int adapter, int64_t f0,
                                         int64_t features, int j0, int lane) {
        const int jj = j0 + 4 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int64_t f = f0 + 16 * h + 8 * r + (lane >> 2);
                const int64_t o = adapter * e.sa + (f < features ? f : features - 1) * e.sf;
                float* to = x[h][r];
                if (e.vec) {
                    uint2 u = make_uint2(0u, 0u);
                    if (jj < e.rank)                     // (the rank is a multiple of 8)
                        u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(e.F) + o + jj));
                    const float2 p = pair16(u.x, e.dtype), q = pair16(u.y, e.dtype);
                    to[0] = p.x;
                    to[1] = p.y;
                    to[2] = q.x;
                    to[3] = q.y;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        to[i] = jj + i < e.rank ? factor_at(e.F, e.dtype, o + (jj + i) * e.sj) : 0.0f;
                }
            }
        a = adapter;
        j = j0;
    }
};

// A tile's rows of T and its tokens' adapters in shared memory (T stays in global
// memory where the room is too small for it), and for tiles that mix adapters
// their tokens in groups of up to eight with one adapter.
struct LowRankTile {
    static constexpr int kTokens = 512, kFast = -0x7fffffff - 1;
    int* adapter;            // [kTokens]
    int* key;                // [kTokens]: the adapter, or kFast in a block of eight alike
    int* groups;             // [kTokens]: first place in `sorted` | tokens << 16
    uint16_t* sorted;        // [kTokens]: tokens by adapter
    int* ngroups;
    float* rows;
    uint32_t room;           // bytes for rows
    const float* t;          // row 0 of the tokens in global memory, or NULL: staged
    __device__ __forceinline__ void place(uint8_t* mem, uint32_t bytes) {
        adapter = reinterpret_cast<int*>(mem);           // 16-byte aligned
        key = adapter + kTokens;
        groups = key + kTokens;
        sorted = reinterpret_cast<uint16_t*>(groups + kTokens);
        ngroups = reinterpret_cast<int*>(sorted + kTokens);
        constexpr uint32_t head = kTokens * 14 + 128;
        rows = reinterpret_cast<float*>(mem + head);
        room = bytes - head;
        t = nullptr;
    }
    // tokens m .. m + n - 1, by all `nt` threads of the CTA; the caller synchronises
    // before using them.  Those past M, whose results are not stored, count as the
    // last token's neighbours (their staged rows hold anything); where T is not
    // staged they have no adapter, so that no row past M is read.
    __device__ __forceinline__ void stage(const LowRankEpi& e, int64_t m, int n, int64_t M, int tid,
                                          int nt) {
        const bool fits = (uint32_t)(n * e.ld) * 4u <= room;
        for (int i = tid; i < n; i += nt) {
            const int64_t at = m + i < M ? m + i : fits && m < M ? M - 1 : -1;
            adapter[i] = at >= 0 ? lowrank_adapter(e, at) : -1;
        }
        if (tid == 0) *ngroups = 0;
        const int per = e.ld >> 2;                       // float4s a row
        t = e.T + m * e.ld;
        if (fits) {
            const int64_t have = (M - m) * per;
            const int all = n * per < have ? n * per : (int)have;
#pragma unroll 4
            for (int i = tid; i < all; i += nt)
                reinterpret_cast<float4*>(rows)[i] = __ldcg(reinterpret_cast<const float4*>(t) + i);
            t = nullptr;
        }
    }
    // whether tokens c .. c + 7 are staged and have one adapter (or none) in common
    __device__ __forceinline__ bool fast(int c) const {
        if (t != nullptr) return false;
        const int4 a0 = *reinterpret_cast<const int4*>(adapter + c);
        const int4 a1 = *reinterpret_cast<const int4*>(adapter + c + 4);
        return a0.y == a0.x && a0.z == a0.x && a0.w == a0.x && a1.x == a0.x && a1.y == a0.x &&
               a1.z == a0.x && a1.w == a0.x;
    }
    // key[] of token i; whether its block is one to be grouped
    __device__ __forceinline__ bool mark(int i) {
        const bool f = fast(i & ~7);
        key[i] = f ? kFast : adapter[i];
        return !f;
    }
    // Sort those of the n tokens (a multiple of 8) that are not in fast blocks into
    // groups of one adapter, by all nt threads; the caller synchronises before and
    // after.  The order of the groups is not fixed, and no result depends on it.
    __device__ __forceinline__ void group(int n, int tid, int nt) {
        for (int i = tid; i < n; i += nt) {
            const int a = key[i];
            if (a == kFast) continue;
            int less = 0, before = 0, same = 0;
#pragma unroll 2
            for (int j = 0; j < n; j += 4) {
                const int4 o = *reinterpret_cast<const int4*>(key + j);
                less += (o.x < a) + (o.y < a) + (o.z < a) + (o.w < a);
                same += (o.x == a) + (o.y == a) + (o.z == a) + (o.w == a);
                before += (o.x == a && j < i) + (o.y == a && j + 1 < i) + (o.z == a && j + 2 < i) +
                          (o.w == a && j + 3 < i);
            }
            sorted[less + before] = (uint16_t)i;
            if ((before & 7) == 0) {
                const int left = same - before;
                groups[atomicAdd(ngroups, 1)] = (less + before) | ((left < 8 ? left : 8) << 16);
            }
        }
    }
    // v[h][e] += ranks j .. j + 15 of the terms of eight tokens with adapter a at the
    // warp's 32 features from f0, in the layout of an m16n8 MMA: feature 16 h + lane / 4 +
    // 8 (e / 2), token 2 (lane % 4) + e % 2; `tok` is the lane's token lane / 4 (-1:
    // absent).  tf32 MMAs: T is split into two tf32 halves and so are fp32 factors
    // (16-bit ones are exact), which leaves below 2^-21 of a product; the sum starts
    // at 0 and is added to v with one rounding.
    __device__ __forceinline__ void add_block(const LowRankEpi& e, LowRankFrag& r, int a, int tok, int j,
                                              int64_t f0, int64_t features, int lane,
                                              float (&v)[2][4]) const {
        if (r.a != a || r.j != j) r.load(e, a, f0, features, j, lane);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tok >= 0) {
            if (t == nullptr) x = *reinterpret_cast<const float4*>(rows + tok * e.ld + j + 4 * (lane & 3));
            else x = __ldcg(reinterpret_cast<const float4*>(t + (int64_t)tok * e.ld + j + 4 * (lane & 3)));
        }
        uint32_t hi[4], lo[4];
        split_tf32(x.x, hi[0], lo[0]);
        split_tf32(x.y, hi[1], lo[1]);
        split_tf32(x.z, hi[2], lo[2]);
        split_tf32(x.w, hi[3], lo[3]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                const float* y0 = r.x[h][0] + 2 * kb;
                const float* y1 = r.x[h][1] + 2 * kb;
                uint32_t q0 = __float_as_uint(y0[0]), q1 = __float_as_uint(y1[0]);
                uint32_t q2 = __float_as_uint(y0[1]), q3 = __float_as_uint(y1[1]);
                if (e.dtype == 2) {
                    uint32_t l0, l1, l2, l3;
                    split_tf32(y0[0], q0, l0);
                    split_tf32(y1[0], q1, l1);
                    split_tf32(y0[1], q2, l2);
                    split_tf32(y1[1], q3, l3);
                    mma_tf32(d, l0, l1, l2, l3, hi[2 * kb], hi[2 * kb + 1]);
                }
                mma_tf32(d, q0, q1, q2, q3, lo[2 * kb], lo[2 * kb + 1]);
                mma_tf32(d, q0, q1, q2, q3, hi[2 * kb], hi[2 * kb + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = __fadd_rn(v[h][i], d[i]);
        }
    }
};

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

// The terms of one token (clamped to M - 1) at two features, without branches, so
// that the loads of several tokens are in flight together.
__device__ __forceinline__ float2 lowrank_pair(const LowRankEpi& e, int64_t m, int64_t M, int64_t f0,
                                               int64_t f1) {
    const int64_t mc = m < M ? m : M - 1;
    const int a = lowrank_adapter(e, mc), ac = a < 0 ? 0 : a;
    float2 d = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int j = 0; j < e.ld; j += 16) {
        float2 b0[8], b1[8];
        lowrank_load16(e, ac, f0, j, b0);
        lowrank_load16(e, ac, f1, j, b1);
        d.x = __fadd_rn(d.x, lowrank_dot16(e.T + mc * e.ld + j, b0));
        d.y = __fadd_rn(d.y, lowrank_dot16(e.T + mc * e.ld + j, b1));
    }
    // (a token without an adapter has read a row that nothing wrote)
    return a < 0 ? make_float2(0.0f, 0.0f) : d;
}

}  // namespace hqq
