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
// One cluster of C CTAs (C = 1 for up to 32768 16-bit logits) owns a token: the
// row is read once into registers, each thread keeps a running maximum and sum
// of exponentials, the pairs are joined by shuffles, shared memory and (C > 1)
// distributed shared memory, and the gradient is formed from the same
// registers, so a pass moves V elements in and V out and is bound by HBM.
// Rows too long for eight CTAs' registers are read a second time instead.
// The K entries are handled beside the dense row: one warp computes p, and after
// the dense gradient is stored each distinct index is overwritten with the full
// expression (one rounding to the output type; duplicates are summed in entry
// order, so results do not depend on any execution order).
// All arithmetic is in fp32; exponentials are ex2.approx of (z - max) log2(e)/t,
// formed from the exact difference so that rows of equal values of any size
// (masks at a type's lowest value) stay finite.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "hqq_params.cuh"

namespace cg = cooperative_groups;

namespace hqq {

namespace {

constexpr int kDsThreads = 512;
constexpr int kDsWarps = kDsThreads / 32;
constexpr int kDsMaxCluster = 8;

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

// W consecutive values of a row: 16 bytes, or one element.
template <typename T, int W>
struct alignas(sizeof(T) * W) Pack {
    T v[W];
};

template <typename T, int W>
__device__ __forceinline__ Pack<T, W> load_pack(const T* p) {
    Pack<T, W> r;
    if constexpr (sizeof(T) * W == 16) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        r = *reinterpret_cast<const Pack<T, W>*>(&u);
    } else {
        r.v[0] = *p;
    }
    return r;
}

template <typename T, int W>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, W>& r) {
    if constexpr (sizeof(T) * W == 16)
        __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&r));
    else
        *p = r.v[0];
}

// Pack i of a row of V values: the last one may be partial (-inf beyond V).
template <typename T, int W>
__device__ __forceinline__ Pack<T, W> row_pack(const T* row, int64_t i, int64_t V) {
    if (W == 1 || (i + 1) * W <= V) return load_pack<T, W>(row + i * W);
    Pack<T, W> r;
#pragma unroll
    for (int e = 0; e < W; ++e)
        r.v[e] = i * W + e < V ? row[i * W + e] : from_float<T>(-INFINITY);
    return r;
}

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
template <typename T, int W>
__device__ __forceinline__ void exps(const Pack<T, W>& z, float m, float c, float2 (&e)[(W + 1) / 2]) {
    if constexpr (W == 1) {
        e[0].x = ex2(__fmul_rn(__fsub_rn(as_float(z.v[0]), m), c));
        e[0].y = 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const float2 d = __fmul2_rn(
                __fadd2_rn(make_float2(as_float(z.v[i]), as_float(z.v[i + 1])), make_float2(-m, -m)),
                make_float2(c, c));
            e[i / 2] = make_float2(ex2(d.x), ex2(d.y));
        }
    }
}

// The largest value of N packs (NaN is passed over: it shows in the sum).
template <typename T, int W, int N>
__device__ __forceinline__ float pack_max(const Pack<T, W> (&z)[N]) {
    if constexpr (W == 1 || sizeof(T) == 4) {
        float mx = as_float(z[0].v[0]);
#pragma unroll
        for (int u = 0; u < N; ++u)
#pragma unroll
            for (int e = 0; e < W; ++e) mx = fmaxf(mx, as_float(z[u].v[e]));
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
template <typename T, int W, int N>
__device__ __forceinline__ void local_stats(const Pack<T, W> (&z)[N], float c, float& m, float& s) {
    const float mx = fmaxf(m, pack_max(z));
    const float base = mx == -INFINITY ? 0.0f : mx;
    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < N; ++u) {
        float2 e[(W + 1) / 2];
        exps(z[u], base, c, e);
#pragma unroll
        for (int i = 0; i < (W + 1) / 2; ++i) acc = __fadd2_rn(acc, e[i]);
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
// row is at most kDsThreads * NV packs and stays in registers.
template <typename T, int W, int NV, bool CACHED>
__global__ void __launch_bounds__(kDsThreads, 2)
distill_kernel(const __grid_constant__ DistillParams p, int csize) {
    __shared__ float st[kDistillMaxTop], sz[kDistillMaxTop];   // teacher value, student logit
    __shared__ int4 si4[kDistillMaxTop / 4];                   // index, or -1
    __shared__ float wm[kDsWarps], ws[kDsWarps], tm_w[kDsWarps], ts_w[kDsWarps], loss_w[kDsWarps];
    __shared__ float cm[kDsMaxCluster], cs[kDsMaxCluster];
    int* si = reinterpret_cast<int*>(si4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = csize == 1 ? 0 : (int)(blockIdx.x % (unsigned)csize);
    const int64_t tok = csize == 1 ? (int64_t)blockIdx.x : (int64_t)(blockIdx.x / (unsigned)csize);
    const T* row = static_cast<const T*>(p.logits) + tok * p.logits_stride;
    T* grow = p.grad ? static_cast<T*>(p.grad) + tok * p.grad_stride : nullptr;
    const float w = p.weight ? p.weight[tok] : 1.0f;
    const float c = p.log2e_t;                           // log2(e) / t
    const int64_t packs = (p.V + W - 1) / W;
    const int64_t lo = packs * rank / csize, hi = packs * (rank + 1) / csize;

    if (w == 0.0f) {                                     // (every CTA of the cluster)
        if (grow) {
            Pack<T, W> zero;
#pragma unroll
            for (int e = 0; e < W; ++e) zero.v[e] = from_float<T>(0.0f);
            for (int64_t i = lo + tid; i < hi; i += kDsThreads) {
                if (W == 1 || (i + 1) * W <= p.V) store_pack<T, W>(grow + i * W, zero);
                else
                    for (int e = 0; i * W + e < p.V; ++e) grow[i * W + e] = zero.v[e];
            }
        }
        if (rank == 0 && tid == 0) {
            if (p.loss) p.loss[tok] = 0.0f;
            if (p.lse) p.lse[tok] = 0.0f;
        }
        return;
    }
    if (csize > 1)                                       // every CTA has started (waited below)
        asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

    Pack<T, W> z[NV];
    auto load_round = [&](int64_t i0) {
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const int64_t i = i0 + (int64_t)u * kDsThreads;
            if (i < hi) {
                z[u] = row_pack<T, W>(row, i, p.V);
            } else {
#pragma unroll
                for (int e = 0; e < W; ++e) z[u].v[e] = from_float<T>(-INFINITY);
            }
        }
    };
    if constexpr (CACHED) load_round(lo + tid);          // in flight behind the entries' loads

    // ---- the teacher's entries, one a thread (two from 512 entries on): value,
    // index and the student's logit there (rank 0 needs all of them for the loss,
    // the others their own segment's), (maximum, sum) as for the row
    const int64_t seg0 = lo * W, seg1 = hi * W;
    float tm = -INFINITY, ts = 0.0f;
    for (int k = tid; k < p.K; k += kDsThreads) {
        const int64_t at = p.at64 ? static_cast<const int64_t*>(p.at)[tok * p.K + k]
                                  : (int64_t) static_cast<const int32_t*>(p.at)[tok * p.K + k];
        const float t0 = load_top(p, tok * p.K + k);
        const bool ok = at >= 0 && at < p.V;
        const float t = ok ? t0 : -INFINITY;
        si[k] = ok ? (int)at : -1;
        st[k] = t;
        sz[k] = ok && (rank == 0 || (at >= seg0 && at < seg1)) ? as_float(row[at]) : 0.0f;
        const float mx = fmaxf(tm, t), base = mx == -INFINITY ? 0.0f : mx;
        ts = __fadd_rn(__fmul_rn(ts, tm == -INFINITY ? 1.0f : ex2(__fmul_rn(__fsub_rn(tm, base), c))),
                       ex2(__fmul_rn(__fsub_rn(t, base), c)));
        tm = mx;
    }
    if (tid < 4 && p.K + tid < ((p.K + 3) & ~3)) si[p.K + tid] = -1;   // the last int4

    // ---- maximum and sum of exponentials of the row
    float m = -INFINITY, s = 0.0f;
    if constexpr (CACHED) {
        local_stats(z, c, m, s);
    } else {
        for (int64_t i0 = lo + tid; i0 < hi; i0 += (int64_t)NV * kDsThreads) {
            load_round(i0);
            local_stats(z, c, m, s);
        }
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
        for (int64_t i0 = lo + tid; i0 < hi; i0 += (int64_t)NV * kDsThreads) {
#pragma unroll
            for (int u = 0; u < NV; ++u) {
                const int64_t i = i0 + (int64_t)u * kDsThreads;
                if (i < hi) {
                    Pack<T, W> q;
                    float2 e[(W + 1) / 2];
                    if constexpr (CACHED) q = z[u];
                    else q = row_pack<T, W>(row, i, p.V);
                    exps(q, m, c, e);
#pragma unroll
                    for (int j = 0; j < (W + 1) / 2; ++j) {
                        e[j] = __fmul2_rn(e[j], make_float2(coef, coef));
                        q.v[2 * j] = from_float<T>(e[j].x);
                        if constexpr (W > 1) q.v[2 * j + 1] = from_float<T>(e[j].y);
                    }
                    if (W == 1 || (i + 1) * W <= p.V) {
                        store_pack<T, W>(grow + i * W, q);
                    } else {
#pragma unroll
                        for (int j = 0; j < W; ++j)
                            if (i * W + j < p.V) grow[i * W + j] = q.v[j];
                    }
                }
            }
            if constexpr (CACHED) break;
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
        int same = 0;                                    // entries of this index
#pragma unroll 4
        for (int j = 0; j < (p.K + 3) / 4; ++j) {
            const int4 o = si4[j];
            same += (o.x == at) + (o.y == at) + (o.z == at) + (o.w == at);
        }
        float mass = mass_of(k);
        if (same > 1) {                                  // in entry order; the first writes
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

template <typename T, int W, int NV, bool CACHED>
cudaError_t launch_ds(const DistillParams& p, int csize, cudaStream_t stream) {
    auto kern = distill_kernel<T, W, NV, CACHED>;
    if (csize == 1) {
        kern<<<(unsigned)p.T, kDsThreads, 0, stream>>>(p, 1);
        return cudaGetLastError();
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)csize;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(p.T * csize));
    cfg.blockDim = dim3(kDsThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p, csize);
}

template <typename T, int W, int NV>
cudaError_t launch_w(const DistillParams& p, cudaStream_t stream) {
    constexpr int64_t kCap = (int64_t)kDsThreads * NV * W;      // values a CTA caches
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int csize = 1;
    // (a share is at most ceil(packs / csize) packs)
    while (csize < kDsMaxCluster && csize * kCap < p.V) csize *= 2;
    // few tokens: more CTAs per row while the grid is short of one per SM and
    // every thread keeps two packs
    while (csize < kDsMaxCluster && p.T * csize * 2 <= sms && p.V >= (int64_t)4 * csize * kDsThreads * W)
        csize *= 2;
    return csize * kCap >= p.V ? launch_ds<T, W, NV, true>(p, csize, stream)
                               : launch_ds<T, W, NV, false>(p, csize, stream);
}

template <typename T>
cudaError_t launch_t(const DistillParams& p, cudaStream_t stream) {
    constexpr int W = 16 / (int)sizeof(T);
    const bool vec = (reinterpret_cast<uintptr_t>(p.logits) & 15u) == 0 && p.logits_stride % W == 0 &&
                     (!p.grad || ((reinterpret_cast<uintptr_t>(p.grad) & 15u) == 0 &&
                                  p.grad_stride % W == 0));
    return vec ? launch_w<T, W, 8>(p, stream) : launch_w<T, 1, 32>(p, stream);
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
