// hqq_distill.cu -- distillation loss of a quantized (student) model against a
// teacher's stored top logits, and its gradient with respect to the logits.
//
// Per token, with z = logits / t over the vocabulary, the teacher's entries
// (value, index) k = 1..K at the same temperature t, weight w:
//   p_k  = exp(top_k / t - L),  L = the teacher's log-sum-exp: given, or taken
//          over the valid entries (0 <= index < vocab);
//   loss = w sum_k p_k (log p_k - log softmax(z)[index_k]);
//   grad[v] = (w / t) (sum_k p_k  softmax(z)[v] - sum_{k: index_k = v} p_k).
//
// One cluster of C CTAs owns a token.  A CTA's share of the row (up to 64 KiB, three
// CTAs per SM) is brought into shared memory by one bulk copy, so the copies of
// one token run beside the arithmetic of the others on the SM; two passes over it
// follow: running maximum and sum of exponentials (joined by shuffles, shared
// memory and, C > 1, distributed shared memory), then the gradient.  A pass moves
// V elements in and V out: the bound is HBM, with the exponentials' instructions
// and the special-function pipe close behind: 4096 x 32000 fp16, 64 entries, a quarter
// of weight 0: 100 us, 4.6 TB/s (rows in registers of two CTAs per SM: 168 us); 2048 x
// 131072 bf16, 256 entries: 286 us, 3.8 TB/s (repeated indices sought by comparing
// all pairs: 481 us).  Rows longer than eight CTAs' shared memory
// are read a second time instead.  Rows off 16 bytes are handled as the aligned
// 16-byte packs that cover them, the elements outside masked.
// The K entries are handled beside the dense row: a thread takes an entry's value
// and the student's logit, and after the dense gradient is stored each distinct
// index is overwritten with the full expression (one rounding to the output type;
// duplicates are summed in entry order, so results do not depend on any
// execution order).
// All arithmetic is in fp32; exponentials are ex2.approx of (z - max) log2(e)/t,
// formed from the exact difference so that rows of equal values of any size
// (masks at a type's lowest value) stay finite.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "hqq_tcgen05.cuh"

namespace cg = cooperative_groups;

namespace hqq {

namespace {

constexpr int kDsThreads = 256;
constexpr int kDsWarps = kDsThreads / 32;
constexpr int kDsMaxCluster = 8;
constexpr int kDsTries = 1000;                  // of the wait for the row before it is timed
constexpr int64_t kDsMaxShare = 196608;          // bytes of a row kept by one CTA

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T> __device__ __forceinline__ float as_float(T v);
template <> __device__ __forceinline__ float as_float(float v) { return v; }
template <> __device__ __forceinline__ float as_float(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float as_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_float(float v);
template <> __device__ __forceinline__ float from_float(float v) { return v; }
template <> __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }

// 16 bytes of a row.
template <typename T>
struct alignas(16) Pack {
    static constexpr int W = 16 / (int)sizeof(T);
    T v[W];
    // values 2 i and 2 i + 1, converted a word at a time
    __device__ __forceinline__ float2 pair(int i) const {
        if constexpr (sizeof(T) == 4) {
            return make_float2(v[2 * i], v[2 * i + 1]);
        } else {
            const uint32_t u = reinterpret_cast<const uint32_t*>(v)[i];
            if constexpr (std::is_same<T, __half>::value)
                return __half22float2(*reinterpret_cast<const __half2*>(&u));
            else
                return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    }
    __device__ __forceinline__ void set_pair(int i, float2 x) {
        if constexpr (sizeof(T) == 4) {
            v[2 * i] = x.x;
            v[2 * i + 1] = x.y;
        } else if constexpr (std::is_same<T, __half>::value) {
            reinterpret_cast<__half2*>(v)[i] = __floats2half2_rn(x.x, x.y);
        } else {
            reinterpret_cast<__nv_bfloat162*>(v)[i] = __floats2bfloat162_rn(x.x, x.y);
        }
    }
};

// The joined (maximum, sum of exponentials relative to it) of the warp's lanes,
// in a fixed order; lanes without values hold (-inf, 0).  A maximum of -inf
// keeps the plain sum (0, or the NaN of a value).
template <int LANES>
__device__ __forceinline__ void join_lanes(float& m, float& s, float c) {
    float mm = m;
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
    s = __fmul_rn(s, mm == -INFINITY ? 1.0f : ex2(__fmul_rn(__fsub_rn(m, mm), c)));
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, o));
    m = mm;
}

// The exponentials of a pack relative to m: e[i] = 2^((z_i - m) c).
template <typename T>
__device__ __forceinline__ void exps(const Pack<T>& z, float m, float c, float2 (&e)[Pack<T>::W / 2]) {
#pragma unroll
    for (int i = 0; i < Pack<T>::W / 2; ++i) {
        const float2 d = __fmul2_rn(__fadd2_rn(z.pair(i), make_float2(-m, -m)), make_float2(c, c));
        e[i] = make_float2(ex2(d.x), ex2(d.y));
    }
}

// The largest value of N packs (NaN is passed over: it shows in the sum).
template <typename T, int N>
__device__ __forceinline__ float pack_max(const Pack<T> (&z)[N]) {
    constexpr int W = Pack<T>::W;
    if constexpr (sizeof(T) == 4) {
        float mx = z[0].v[0];
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int e = 0; e < W; ++e) mx = fmaxf(mx, z[u].v[e]);
        return mx;
    } else {                                             // two 16-bit values an operation
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2,
                                             __nv_bfloat162>::type;
        T2 mx = *reinterpret_cast<const T2*>(&z[0].v[0]);
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int e = 0; e < W; e += 2)
                mx = __hmax2(mx, *reinterpret_cast<const T2*>(&z[u].v[e]));
        return fmaxf(as_float(mx.x), as_float(mx.y));
    }
}

// Running maximum and sum of a thread, N packs further.
template <typename T, int N>
__device__ __forceinline__ void local_stats(const Pack<T> (&z)[N], float c, float& m, float& s) {
    const float mx = fmaxf(m, pack_max(z));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float2 e[Pack<T>::W / 2];
        exps(z[u], base, c, e);
#pragma unroll
        for (int i = 0; i < Pack<T>::W / 2; ++i) acc = __fadd2_rn(acc, e[i]);
    }
    const float sum = __fadd_rn(acc.x, acc.y);
    // what came before (m, s), relative to the new maximum
    s = m == -INFINITY ? __fadd_rn(s, sum)
                       : __fmaf_rn(s, ex2(__fmul_rn(__fsub_rn(m, base), c)), sum);
    m = mx;
}

__device__ __forceinline__ float load_top(const DistillParams& p, int64_t i) {
    switch (p.top_dtype) {
        case 0: return __half2float(static_cast<const __half*>(p.top)[i]);
        case 1: return __bfloat162float(static_cast<const __nv_bfloat16*>(p.top)[i]);
        default: return static_cast<const float*>(p.top)[i];
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Grid: one cluster of `csize` CTAs per token.  CACHED: the CTA's share of the
// row (at most share_packs packs) is kept in shared memory.
template <typename T, bool CACHED>
__global__ void __launch_bounds__(kDsThreads, 3)
distill_kernel(const __grid_constant__ DistillParams p, int csize, int share_packs) {
    constexpr int W = Pack<T>::W;
    extern __shared__ __align__(16) uint8_t ds_smem[];
    __shared__ float wm[kDsWarps], ws[kDsWarps], tm_w[kDsWarps], ts_w[kDsWarps], loss_w[kDsWarps];
    __shared__ float cm[kDsMaxCluster], cs[kDsMaxCluster];
    __shared__ uint64_t bar;
    __shared__ int abort_flag, repeated;
    Pack<T>* cache = reinterpret_cast<Pack<T>*>(ds_smem);
    // the teacher's entries behind the row: index (or -1), value, student's logit
    int* si = reinterpret_cast<int*>(ds_smem + (CACHED ? (size_t)share_packs * 16 : 0));
    float* st = reinterpret_cast<float*>(si + p.K);
    float* sz = st + p.K;
    int* seen = reinterpret_cast<int*>(sz + p.K);        // hash set of the indices

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = csize == 1 ? 0 : (int)(blockIdx.x % (unsigned)csize);
    const int64_t tok = csize == 1 ? (int64_t)blockIdx.x : (int64_t)(blockIdx.x / (unsigned)csize);
    const T* row = static_cast<const T*>(p.logits) + tok * p.logits_stride;
    T* grow = p.grad ? static_cast<T*>(p.grad) + tok * p.grad_stride : nullptr;
    const float w = p.weight ? p.weight[tok] : 1.0f;
    const float c = p.log2e_t;                           // log2(e) / t
    // the aligned packs that cover the row: `head` elements before it in the first
    const int head = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const Pack<T>* packs = reinterpret_cast<const Pack<T>*>(row - head);
    // (below 2^31 elements: counts of packs fit 32 bits)
    const int np = (int)((p.V + head + W - 1) / W);
    const int lo = (int)((int64_t)np * rank / csize), hi = (int)((int64_t)np * (rank + 1) / csize);
    // the row's elements [seg0, seg1) that this CTA owns
    const int64_t seg0 = lo == 0 ? 0 : (int64_t)lo * W - head;
    const int64_t seg1 = hi == np ? p.V : (int64_t)hi * W - head;
    // packs wholly inside the row; the others are the owning threads' extra work
    const int in0 = lo == 0 && head ? 1 : lo;
    const int in1 = hi == np && (p.V + head) % W ? hi - 1 : hi;
    // gradient rows of the same alignment are stored in whole packs
    const bool whole = grow && (reinterpret_cast<uintptr_t>(grow) & 15u) / sizeof(T) == (unsigned)head;
    uint4* gpacks = reinterpret_cast<uint4*>(grow - head);
    auto store_each = [&](int i, const Pack<T>& q) {     // pack i, elements of the row alone
        const int64_t e0 = (int64_t)i * W - head;
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e0 + e >= 0 && e0 + e < p.V) grow[e0 + e] = q.v[e];
    };
    auto store = [&](int i, const Pack<T>& q) {
        if (whole && i >= in0 && i < in1) __stcs(gpacks + i, *reinterpret_cast<const uint4*>(&q));
        else store_each(i, q);
    };

    if (w == 0.0f) {                                     // (every CTA of the cluster)
        if (grow) {
            Pack<T> zero;
#pragma unroll
            for (int e = 0; e < W; ++e) zero.v[e] = from_float<T>(0.0f);
            for (int i = lo + tid; i < hi; i += kDsThreads) store(i, zero);
        }
        if (rank == 0 && tid == 0) {
            if (p.loss) p.loss[tok] = 0.0f;
            if (p.lse) p.lse[tok] = 0.0f;
        }
        return;
    }
    if (csize > 1)                                       // every CTA has started (waited below)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (tid == 0) {
        abort_flag = 0;
        repeated = 0;
        if constexpr (CACHED) {
            mbar_init(smem_u32(&bar), 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            const uint32_t bytes = (uint32_t)(hi - lo) * 16u;
            mbar_expect_tx(smem_u32(&bar), bytes);
            if (bytes)
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
                        "r"(smem_u32(ds_smem)), "l"(packs + lo), "r"(bytes), "r"(smem_u32(&bar))
                    : "memory");
        }
    }
    for (int i = tid; i <= p.hash_mask; i += kDsThreads) seen[i] = -1;
    __syncthreads();                                     // barrier and hash set are ready
    // pack i with the elements outside the row -inf
    auto masked = [&](int i, Pack<T> q) {
        const int64_t e0 = (int64_t)i * W - head;
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e0 + e < 0 || e0 + e >= p.V) q.v[e] = from_float<T>(-INFINITY);
        return q;
    };
    auto load = [&](int i) {
        if constexpr (CACHED) {
            return cache[i - lo];                        // (masked there once)
        } else {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(packs + i));
            const Pack<T> q = *reinterpret_cast<const Pack<T>*>(&u);
            return i >= in0 && i < in1 ? q : masked(i, q);
        }
    };

    // ---- the teacher's entries, one a thread and round: value,
    // index and the student's logit there (rank 0 needs all of them for the loss,
    // the others their own segment's), (maximum, sum) as for the row
    float tm = -INFINITY, ts = 0.0f;
    for (int k = tid; k < p.K; k += kDsThreads) {
        const int64_t at = p.at64 ? static_cast<const int64_t*>(p.at)[tok * p.K + k]
                                  : (int64_t) static_cast<const int32_t*>(p.at)[tok * p.K + k];
        const float t0 = load_top(p, tok * p.K + k);
        const bool ok = at >= 0 && at < p.V;
        const float t = ok ? t0 : -INFINITY;
        si[k] = ok ? (int)at : -1;
        st[k] = t;
        const bool mine = ok && at >= seg0 && at < seg1;
        sz[k] = mine || (ok && rank == 0) ? as_float(row[at]) : 0.0f;
        if (mine && grow) {                              // an index met twice?
            uint32_t h = ((uint32_t)at * 2654435761u) >> 20;
            for (int n = 0; n <= p.hash_mask; ++n, ++h) {
                const int old = atomicCAS(seen + (h & (uint32_t)p.hash_mask), -1, (int)at);
                if (old == -1) break;
                if (old == (int)at) {
                    repeated = 1;
                    break;
                }
            }
        }
        const float mx = fmaxf(tm, t), base = mx == -INFINITY ? 0.0f : mx;
        ts = __fadd_rn(__fmul_rn(ts, tm == -INFINITY ? 1.0f : ex2(__fmul_rn(__fsub_rn(tm, base), c))),
                       ex2(__fmul_rn(__fsub_rn(t, base), c)));
        tm = mx;
    }

    // ---- maximum and sum of exponentials of the row, four packs at a time
    float m = -INFINITY, s = 0.0f;
    if constexpr (CACHED) {
        bool landed = false;
        for (int i = 0; i < kDsTries && !landed; ++i) landed = mbar_try(smem_u32(&bar), 0u);
        if (!landed && !mbar_wait(smem_u32(&bar), 0u, &abort_flag, nullptr, true)) {
            // the row did not arrive in time: no value of it is to be trusted, and NaN in
            // one CTA's sum is NaN in every output of the token; the copy gets the same
            // time once more before the CTA can end
            s = __int_as_float(0x7fffffff);
            mbar_wait(smem_u32(&bar), 0u, &abort_flag, nullptr, true);
        }
    }
    if constexpr (CACHED) {
        // the packs at the row's ends, by the threads that own them in both passes
        if (in0 > lo && tid == 0) cache[0] = masked(lo, cache[0]);
        if (in1 < hi && tid == (hi - 1 - lo) % kDsThreads) cache[hi - 1 - lo] = masked(hi - 1, cache[hi - 1 - lo]);
    }
    int i0 = lo + tid;
    for (; i0 + 3 * kDsThreads < hi; i0 += 4 * kDsThreads) {
        Pack<T> z[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) z[u] = load(i0 + u * kDsThreads);
        local_stats(z, c, m, s);
    }
    for (; i0 < hi; i0 += kDsThreads) {
        Pack<T> z[1] = {load(i0)};
        local_stats(z, c, m, s);
    }
    join_lanes<32>(m, s, c);
    if (warp * 32 < p.K) join_lanes<32>(tm, ts, c);
    if (lane == 0) {
        wm[warp] = m;
        ws[warp] = s;
        tm_w[warp] = tm;                                 // (-inf, 0) where there are no entries
        ts_w[warp] = ts;
    }
    __syncthreads();
    m = wm[lane % kDsWarps];
    s = ws[lane % kDsWarps];
    tm = tm_w[lane % kDsWarps];
    ts = ts_w[lane % kDsWarps];
    join_lanes<kDsWarps>(m, s, c);
    join_lanes<kDsWarps>(tm, ts, c);
    if (csize > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (tid < csize) {
            *cluster.map_shared_rank(&cm[rank], tid) = m;
            *cluster.map_shared_rank(&cs[rank], tid) = s;
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
        m = lane % kDsMaxCluster < csize ? cm[lane % kDsMaxCluster] : -INFINITY;
        s = lane % kDsMaxCluster < csize ? cs[lane % kDsMaxCluster] : 0.0f;
        join_lanes<kDsMaxCluster>(m, s, c);
    }
    const float logs = logf(s);
    // L, log p_k = t_k / t - L and sum of the p_k (1 up to rounding without a
    // teacher_lse); no entry, or none with mass: L = -inf, sum 0
    const bool given = p.teacher_lse != nullptr;
    const float L = given ? p.teacher_lse[tok] : logf(ts);
    const float toff = given || tm == -INFINITY ? 0.0f : tm;
    auto log_p = [&](float t) { return __fsub_rn(__fmul_rn(__fsub_rn(t, toff), p.inv_t), L); };
    const float psum = tm == -INFINITY ? __fmul_rn(ts, 0.0f)
                       : given ? __fmul_rn(ts, expf(__fsub_rn(__fmul_rn(tm, p.inv_t), L)))
                               : __fdiv_rn(ts, ts);

    // ---- loss (rank 0)
    if (rank == 0 && p.lse && tid == 0) p.lse[tok] = __fadd_rn(__fmul_rn(m, p.inv_t), logs);
    if (rank == 0 && p.loss && warp * 32 < p.K) {
        float acc = 0.0f;
        for (int k = tid; k < p.K; k += kDsThreads) {
            const float t = st[k];
            // entries without mass (unused, or a value of -inf) take no part
            const float lp = log_p(t), pk = t == -INFINITY ? 0.0f : expf(lp);
            if (pk != 0.0f) {                            // (NaN != 0: kept)
                const float lq = __fsub_rn(__fmul_rn(__fsub_rn(sz[k], m), p.inv_t), logs);
                acc = __fmaf_rn(pk, __fsub_rn(lp, lq), acc);
            }
        }
        acc = warp_sum(acc);
        if (lane == 0) loss_w[warp] = acc;
    }

    // ---- gradient: the dense row, then the entries' places
    const float wt = __fmul_rn(w, p.inv_t);
    if (grow) {
        const float coef = __fdiv_rn(__fmul_rn(wt, psum), s);
        auto gradient = [&](Pack<T> q) {
            float2 e[W / 2];
            exps(q, m, c, e);
#pragma unroll
            for (int j = 0; j < W / 2; ++j)
                q.set_pair(j, __fmul2_rn(e[j], make_float2(coef, coef)));
            return q;
        };
        if (whole) {
            int i = lo + tid;
            if (i < in0) {
                store_each(i, gradient(load(i)));
                i += kDsThreads;
            }
#pragma unroll 2
            for (; i < in1; i += kDsThreads) {
                const Pack<T> q = gradient(load(i));
                __stcs(gpacks + i, *reinterpret_cast<const uint4*>(&q));
            }
            if (i < hi) store_each(i, gradient(load(i)));
        } else {
            for (int i = lo + tid; i < hi; i += kDsThreads) store_each(i, gradient(load(i)));
        }
    }
    __syncthreads();                                     // the dense row is stored
    if (rank == 0 && p.loss && tid == 0) {
        float acc = loss_w[0];
        for (int i = 1; i * 32 < p.K && i < kDsWarps; ++i) acc = __fadd_rn(acc, loss_w[i]);
        p.loss[tok] = __fmul_rn(w, acc);
    }
    if (!grow) return;
    const float coef = __fdiv_rn(__fmul_rn(wt, psum), s);
    auto mass_of = [&](int k) { return st[k] == -INFINITY ? 0.0f : expf(log_p(st[k])); };
    for (int k = tid; k < p.K; k += kDsThreads) {
        const int at = si[k];
        if (at < seg0 || at >= seg1) continue;           // (unused entries: -1)
        float mass = mass_of(k);
        if (repeated) {                                  // in entry order; the first writes
            bool first = true;
            mass = 0.0f;
            for (int j = 0; j < p.K; ++j)
                if (si[j] == at) {
                    if (j < k) first = false;
                    mass = __fadd_rn(mass, mass_of(j));
                }
            if (!first) continue;
        }
        const float e = ex2(__fmul_rn(__fsub_rn(sz[k], m), c));
        grow[at] = from_float<T>(__fmaf_rn(e, coef, -__fmul_rn(wt, mass)));
    }
}

template <typename T, bool CACHED>
cudaError_t launch_ds(const DistillParams& p, int csize, int share_packs, cudaStream_t stream) {
    auto kern = distill_kernel<T, CACHED>;
    const size_t smem = (CACHED ? (size_t)share_packs * 16 : 0) + (size_t)p.K * 12 +
                        (size_t)(p.hash_mask + 1) * 4;
    // the limit is the kernel's, not the call's: one value, the largest, so that calls
    // from several host threads cannot lower it under each other
    constexpr size_t kMost = (CACHED ? (size_t)kDsMaxShare : 0) + (size_t)kDistillMaxTop * (12 + 2 * 4);
    if (smem > kMost) return cudaErrorInvalidValue;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)csize;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(p.T * csize));
    cfg.blockDim = dim3(kDsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = csize > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, p, csize, share_packs);
}

template <typename T>
cudaError_t launch_t(const DistillParams& p, cudaStream_t stream) {
    constexpr int64_t W = Pack<T>::W;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t np = (p.V + 2 * W - 2) / W;            // packs of a row of any alignment
    int csize = 1;
    // a share of 64 KiB at most (three CTAs per SM) while the cluster allows it
    while (csize < kDsMaxCluster && (np + csize - 1) / csize > 65536 / 16) csize *= 2;
    // few tokens: more CTAs per row while the grid is short of one per SM and
    // every thread keeps two packs
    while (csize < kDsMaxCluster && p.T * csize * 2 <= sms && np >= (int64_t)4 * csize * kDsThreads)
        csize *= 2;
    const int64_t share = np / csize + 1;
    return share * 16 <= kDsMaxShare ? launch_ds<T, true>(p, csize, (int)share, stream)
                                     : launch_ds<T, false>(p, csize, 0, stream);
}

}  // namespace

cudaError_t launch_distill(const DistillParams& p, int dtype, cudaStream_t stream) {
    switch (dtype) {
        case 0: return launch_t<__half>(p, stream);
        case 1: return launch_t<__nv_bfloat16>(p, stream);
        case 2: return launch_t<float>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace hqq
