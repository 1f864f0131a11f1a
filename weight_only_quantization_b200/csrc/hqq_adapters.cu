// hqq_adapters.cu -- the products of the low-rank adapters beside a quantized
// linear layer that run outside its main kernels:
//
//   shrink   T[m, :] = s_a A_a X[m]    (and P[m, :] = s_a B_a^T dY[m] for the
//            gradients), a = index[m], fp32 [M, ld] with ld = rank rounded up
//            to 16 and zeros behind the rank;
//   factors  dA_a = sum_{index[m] = a} P[m]^T X[m],
//            dB_a = sum_{index[m] = a} dY[m]^T T[m].
//
// The expanding products (T B^T into Y, P A into dX) are added to the quantized
// product's fp32 accumulators instead (hqq_lowrank_epi.cuh), so the output is
// rounded once and never re-read.
//
// shrink is bound by reading X and the factors (2 r flops a value): a cluster of
// CTAs owns 32 tokens, its warps take interleaved 32-wide steps of the reduction
// and feed warp-level MMAs straight from 16-byte global loads -- a lane's 8
// consecutive k supply two k16 steps, the same permutation of k on both operands
// -- and the partial tiles meet in shared and distributed shared memory.  Tokens
// of different adapters in one tile are separate passes over it (the passes are
// shared out over `slots` clusters), each writing only its own tokens' rows, so
// tokens need no sorting and one token's values never reach another's row.  From
// 257 tokens with several adapters the tiles are taken in the adapters' order all
// the same (1800 tokens of 32 adapters in any order, rank 64, 4096 columns: 133 us
// in the tokens' own order, 31 in the adapters').
// fp16 factors run as fp16 MMAs (products exact in fp32); bf16 and fp32 ones
// as tf32 MMAs, where X and bf16 are exact and fp32 is split into two tf32 halves
// (the dropped part is below 2^-22 of a product).  2048 tokens x 8192, rank 32 in fp32:
// 24 us, where reading X takes 5: latency and the splitting of the factors.
//
// factors: a CTA owns 64 columns of X or dY for one adapter and walks that
// adapter's tokens (listed once per call in token order, no atomics, so the sums
// have a fixed order) in chunks of 64 staged by cp.async; the fp32 operand is split
// into two tf32 halves; each chunk's MMA sums are added to fp32 registers.  2048
// tokens, 8192 + 8192 columns, rank 32: 57 us (70 before the halves were formed by
// integer rounding and the copies' addresses hoisted), bound by instruction issue and
// the tf32 MMAs, not by its 67 MB.
#include <cooperative_groups.h>

#include "hqq_adapters.cuh"
#include "hqq_tf32.cuh"

namespace cg = cooperative_groups;

namespace hqq {

namespace {

constexpr int kShThreads = 256;
constexpr int kShWarps = kShThreads / 32;
constexpr int kShTokens = 32;            // tokens per tile (two m16 blocks)
constexpr int kShMaxCluster = 8;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t half_bits_f32(uint32_t pair, int hi) {
    const __half2 h = *reinterpret_cast<const __half2*>(&pair);
    return __float_as_uint(hi ? __high2float(h) : __low2float(h));
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// A kernel launched beside the one before it does not end before that one: what
// waits for its end may rely on both.
__device__ __forceinline__ void wait_for_prior() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// How a factor's values reach the B operand.
enum FactorForm {
    kKPairs,     // fp16, the reduction index contiguous: one 16-byte load a lane
    kJPairs,     // fp16, the rank contiguous: 8x8 blocks transposed in registers
    kKBf16,      // tf32 MMAs: bf16 or fp32, the reduction index contiguous (16-byte
    kKF32,       //   loads) ..
    kJBf16,      //   .. or the rank contiguous (a sector of 8 or 16 ranks a row)
    kJF32,
    kAnyType     // any type and strides, tf32 MMAs
};

// Grid: x = ((tile * slots) + slot) * csize + cluster rank, y = chunks of 8 NT
// ranks.
template <FactorForm FORM, int NT>
__global__ void __launch_bounds__(kShThreads, 2)
shrink_kernel(const __grid_constant__ ShrinkParams p, int csize, int slots) {
    constexpr int RC = 8 * NT;
    constexpr int TE = kShTokens * RC;                   // values of a tile
    constexpr int PER = (TE + kShThreads - 1) / kShThreads;
    __shared__ float red[kShWarps][TE];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int crank = csize == 1 ? 0 : (int)(blockIdx.x % (unsigned)csize);
    const unsigned cl = csize == 1 ? blockIdx.x : blockIdx.x / (unsigned)csize;
    const int slot = (int)(cl % (unsigned)slots);
    const int64_t m0 = (int64_t)(cl / (unsigned)slots) * kShTokens;
    const int j0 = (int)blockIdx.y * RC;

    // the kernel that reads T may start its own work (it waits for this one's end
    // before it reads)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // the lane's token (-1: past the last) and its adapter (-1: none)
    __shared__ int toks[kShTokens];
    int tok = -1, mine = -1;
    if (m0 + lane < (p.order ? (int64_t)__ldg(p.start + p.count) : p.M))
        tok = p.order ? __ldg(p.order + m0 + lane) : (int)(m0 + lane);
    if (tok >= 0) {
        const int a = p.index ? __ldg(p.index + tok) : 0;
        if ((unsigned)a < (unsigned)p.count) mine = a;
    }
    if (warp == 0) toks[lane] = tok;                     // (read behind a CTA barrier)
    const __half* xr[2][2];                              // rows g, g + 8 of both m16 blocks
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = __shfl_sync(0xffffffffu, tok, 16 * b + 8 * h + g);
            xr[b][h] = p.X + (int64_t)(m < 0 ? 0 : m) * p.ldx + 8 * t;
        }
    const int64_t blocks = (p.K + 31) / 32;
    const int64_t bstep = (int64_t)kShWarps * csize;

    uint32_t todo = __ballot_sync(0xffffffffu, mine >= 0);
    for (int turn = 0; todo; ++turn) {
        const int a = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
        const uint32_t same = __ballot_sync(0xffffffffu, mine == a);
        todo &= ~same;
        if (turn % slots != slot) continue;              // (the same for the whole cluster)
        const bool has[2] = {(same & 0xffffu) != 0, (same >> 16) != 0};
        const int64_t fo = (int64_t)a * p.sa;
        float acc[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[b][n][e] = 0.0f;

#pragma unroll 1
        for (int64_t bl = (int64_t)crank * kShWarps + warp; bl < blocks; bl += bstep) {
            const int64_t k0 = bl * 32, kk = k0 + 8 * t;
            uint4 x[2][2];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    x[b][h] = has[b] && kk < p.K
                                  ? __ldg(reinterpret_cast<const uint4*>(xr[b][h] + k0))
                                  : make_uint4(0u, 0u, 0u, 0u);
            if constexpr (FORM == kKPairs) {
                uint4 f[NT];
                const __half* F = static_cast<const __half*>(p.F) + fo;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int j = j0 + 8 * n + g;
                    f[n] = j < p.rank && kk < p.K
                               ? __ldg(reinterpret_cast<const uint4*>(F + j * p.sj + kk))
                               : make_uint4(0u, 0u, 0u, 0u);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (has[b]) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};       // (as below)
                            mma_f16(d, x[b][0].x, x[b][1].x, x[b][0].y, x[b][1].y, f[n].x, f[n].y);
                            mma_f16(d, x[b][0].z, x[b][1].z, x[b][0].w, x[b][1].w, f[n].z, f[n].w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[b][n][e] = __fadd_rn(acc[b][n][e], d[e]);
                        }
            } else if constexpr (FORM == kJPairs) {
                // slot i of a k16 half is k = 8 (i / 2) + i % 2 (+ 4 for the second
                // MMA, + 2 for its upper half); the lane reads row i = g, ranks 2t, 2t + 1
                const __half* F = static_cast<const __half*>(p.F) + fo;
                uint32_t f[NT][4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int64_t k = k0 + 8 * (g >> 1) + (g & 1) + 2 * (c & 1) + 4 * (c >> 1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = j0 + 8 * n + 2 * t;
                        f[n][c] = j < p.rank && k < p.K
                                      ? __ldg(reinterpret_cast<const uint32_t*>(F + k * p.sk + j))
                                      : 0u;
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) f[n][c] = transpose8x8(f[n][c]);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        if (has[b]) {
                            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};       // (as below)
                            mma_f16(d, x[b][0].x, x[b][1].x, x[b][0].y, x[b][1].y, f[n][0], f[n][1]);
                            mma_f16(d, x[b][0].z, x[b][1].z, x[b][0].w, x[b][1].w, f[n][2], f[n][3]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[b][n][e] = __fadd_rn(acc[b][n][e], d[e]);
                        }
                }
            } else {
                constexpr bool k32 = FORM == kKF32 || FORM == kJF32;
                // the lane's values for each n-tile: rank j0 + 8 n + g, k = kk .. kk + 7
                float v[NT][8];
                if constexpr (FORM == kKBf16 || FORM == kKF32) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = j0 + 8 * n + g;
                        const bool in = j < p.rank && kk < p.K;
                        if constexpr (FORM == kKBf16) {
                            const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(
                                                     static_cast<const __nv_bfloat16*>(p.F) + fo + j * p.sj + kk))
                                               : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                v[n][2 * i] = __uint_as_float(word_of(u, i) << 16);
                                v[n][2 * i + 1] = __uint_as_float(word_of(u, i) & 0xffff0000u);
                            }
                        } else {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float4 u = in ? __ldg(reinterpret_cast<const float4*>(
                                                          static_cast<const float*>(p.F) + fo + j * p.sj + kk) + h)
                                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                v[n][4 * h] = u.x;
                                v[n][4 * h + 1] = u.y;
                                v[n][4 * h + 2] = u.z;
                                v[n][4 * h + 3] = u.w;
                            }
                        }
                    }
                } else if constexpr (FORM == kJBf16 || FORM == kJF32) {
                    const int64_t base = fo + kk * p.sk + j0 + g;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t at = base + i * p.sk;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const bool in = j0 + 8 * n + g < p.rank && kk + i < p.K;
                            if constexpr (FORM == kJF32)
                                v[n][i] = in ? __ldg(static_cast<const float*>(p.F) + at + 8 * n) : 0.0f;
                            else
                                v[n][i] = in ? __bfloat162float(__ldg(
                                                   static_cast<const __nv_bfloat16*>(p.F) + at + 8 * n))
                                             : 0.0f;
                        }
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = j0 + 8 * n + g;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[n][i] = j < p.rank && kk + i < p.K
                                          ? factor_at(p.F, p.dtype, fo + j * p.sj + (kk + i) * p.sk)
                                          : 0.0f;
                    }
                }
                const bool split = k32 || (FORM == kAnyType && p.dtype == 2);
                uint32_t xa[4][2][4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t w0 = word_of(x[b][0], i), w1 = word_of(x[b][1], i);
                        xa[i][b][0] = half_bits_f32(w0, 0);
                        xa[i][b][1] = half_bits_f32(w1, 0);
                        xa[i][b][2] = half_bits_f32(w0, 1);
                        xa[i][b][3] = half_bits_f32(w1, 1);
                    }
                // sums of a step start at 0 and join the running ones with one rounding:
                // an MMA truncates, which over a long chain adds up on one side
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[2][4] = {};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h0 = __float_as_uint(v[n][2 * i]), h1 = __float_as_uint(v[n][2 * i + 1]);
                        uint32_t l0 = 0u, l1 = 0u;
                        if (split) {
                            split_tf32(v[n][2 * i], h0, l0);
                            split_tf32(v[n][2 * i + 1], h1, l1);
                        }
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            if (has[b]) {
                                if (split)
                                    mma_tf32(d[b], xa[i][b][0], xa[i][b][1], xa[i][b][2], xa[i][b][3], l0, l1);
                                mma_tf32(d[b], xa[i][b][0], xa[i][b][1], xa[i][b][2], xa[i][b][3], h0, h1);
                            }
                    }
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[b][n][e] = __fadd_rn(acc[b][n][e], d[b][e]);
                }
            }
        }

        // the warps' partial tiles, then the cluster's (in rank 0's memory)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    red[warp][(16 * b + g + 8 * (e >> 1)) * RC + 8 * n + 2 * t + (e & 1)] =
                        acc[b][n][e];
        __syncthreads();
        float v[PER];
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int e = u * kShThreads + tid;
            v[u] = 0.0f;
            if (TE % kShThreads == 0 || e < TE)
#pragma unroll
                for (int w = 0; w < kShWarps; ++w) v[u] = __fadd_rn(v[u], red[w][e]);
        }
        if (csize > 1) {
            // every CTA has summed its warps: rank 0's buffer is free
            asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                         "barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (crank != 0) {
                float* dst = cg::this_cluster().map_shared_rank(&red[0][0], 0) + (crank - 1) * TE;
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int e = u * kShThreads + tid;
                    if (TE % kShThreads == 0 || e < TE) dst[e] = v[u];
                }
            }
            asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                         "barrier.cluster.wait.acquire.aligned;" ::: "memory");
            if (crank == 0)
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int e = u * kShThreads + tid;
                    if (TE % kShThreads == 0 || e < TE)
                        for (int c = 1; c < csize; ++c)
                            v[u] = __fadd_rn(v[u], (&red[0][0])[(c - 1) * TE + e]);
                }
        }
        if (crank == 0) {
            const float s = p.scaling ? __ldg(p.scaling + a) : 1.0f;
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int e = u * kShThreads + tid;
                const int row = e / RC, j = j0 + e % RC;
                if ((TE % kShThreads == 0 || e < TE) && (same >> row & 1u) && j < p.ld)
                    // (behind the rank: an infinite X times 0 would be NaN)
                    p.T[(int64_t)toks[row] * p.ld + j] = j < p.rank ? __fmul_rn(v[u], s) : 0.0f;
            }
        }
        __syncthreads();                                 // red is written again
    }
    if (p.beside) wait_for_prior();
}

template <FactorForm FORM, int NT>
cudaError_t launch_shrink_nt(const ShrinkParams& p, cudaStream_t stream) {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t tiles = (p.M + kShTokens - 1) / kShTokens;
    const int64_t chunks = (p.ld + 8 * NT - 1) / (8 * NT);
    const int64_t blocks = (p.K + 31) / 32;
    // clusters that share out a tile's adapters: as many as it can hold while the
    // grid is small, few for many tokens (whose tiles rarely mix adapters)
    int64_t slots = p.count < kShTokens ? p.count : kShTokens;
    if (p.M < slots) slots = p.M;
    while (slots > 1 && tiles * slots > 256) slots = (slots + 1) / 2;
    if (p.order && slots > 2) slots = 2;
    // split the reduction while the busy CTAs stay within two per SM and every warp
    // keeps two steps: up to 256 tokens every one may have an adapter of its own, more
    // come as runs of a few
    const int64_t pairs = p.M <= 256 ? (p.M < tiles * slots ? p.M : tiles * slots)
                                     : tiles + (p.index ? p.count : 0);
    int csize = 1;
    while (csize < kShMaxCluster && pairs * chunks * csize <= sms &&
           blocks >= (int64_t)2 * csize * kShWarps)
        csize *= 2;
    auto kern = shrink_kernel<FORM, NT>;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(tiles * slots * csize), (unsigned)chunks);
    cfg.blockDim = dim3(kShThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.beside ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p, csize, (int)slots);
}

template <FactorForm FORM>
cudaError_t launch_shrink_form(const ShrinkParams& p, cudaStream_t stream) {
    return p.ld <= 16 ? launch_shrink_nt<FORM, 2>(p, stream) : launch_shrink_nt<FORM, 4>(p, stream);
}

// ---- the tokens of every adapter, in token order ----------------------------

// Block a lists the tokens of adapter a behind those of the adapters below it:
// start[a] .. start[a + 1] in order[].
__global__ void __launch_bounds__(256)
order_kernel(const int32_t* __restrict__ index, int64_t M, int count, int32_t* __restrict__ order,
             int32_t* __restrict__ start) {
    __shared__ int part[8], below[8];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int a = (int)blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int less = 0;
    for (int64_t m = tid; m < M; m += 256) {
        const int i = __ldg(index + m);
        less += i >= 0 && i < a;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) less += __shfl_xor_sync(0xffffffffu, less, o);
    if (lane == 0) below[warp] = less;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) base += below[w];
    if (tid == 0) start[a] = base;
    for (int64_t m0 = 0; m0 < M; m0 += 256) {
        const int64_t m = m0 + tid;
        const bool in = m < M && __ldg(index + m) == a;
        const uint32_t vote = __ballot_sync(0xffffffffu, in);
        if (lane == 0) part[warp] = __popc(vote);
        __syncthreads();
        int at = base, all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            if (w < warp) at += part[w];
            all += part[w];
        }
        if (in) order[at + __popc(vote & ((1u << lane) - 1u))] = (int32_t)m;
        base += all;
        __syncthreads();
    }
    if (tid == 0 && a == count - 1) start[count] = base;
    wait_for_prior();
}

// ---- gradients of the factors ------------------------------------------------

constexpr int kFgThreads = 256;
constexpr int kFgCols = 64;              // columns of X or dY per CTA
constexpr int kFgTokens = 64;            // tokens per stage
constexpr int kFgStages = 2;
constexpr int kFgMaxCluster = 4;
constexpr int kFgZ = kFgCols + 16;       // halves per staged row: 8 rows apart in the banks

template <int NT>
struct FgGeo {
    static constexpr int RC = 8 * NT;
    static constexpr int SS = RC + 8;    // floats per staged row of T or P
    static constexpr int STAGE = kFgTokens * (kFgZ * 2 + SS * 4);
    static constexpr int RED = 4 * kFgCols * RC * 4;             // the token quarters
    static constexpr int XRED = (kFgMaxCluster - 1) * kFgCols * RC * 4;
    static constexpr int BYTES = kFgStages * STAGE > RED + XRED ? kFgStages * STAGE : RED + XRED;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}

// Grid: x = column tile * csize + cluster rank, y = adapter, z = chunks of 8 NT
// ranks.  Tiles below tiles_a make dA from X and P, the others dB from dY and T.
template <int NT>
__global__ void __launch_bounds__(kFgThreads, NT <= 4 ? 3 : 2)
factor_grad_kernel(const __grid_constant__ FactorGradParams p, int csize) {
    using G = FgGeo<NT>;
    constexpr int RC = G::RC;
    extern __shared__ __align__(16) uint8_t fg_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    const int crank = csize == 1 ? 0 : (int)(blockIdx.x % (unsigned)csize);
    const int tile = (int)(csize == 1 ? blockIdx.x : blockIdx.x / (unsigned)csize);
    // (the input gradient's kernel may start its own work)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    wait_for_prior();                                    // T, P and the lists are there
    const int a = (int)blockIdx.y, j0 = (int)blockIdx.z * RC;
    const bool isA = tile < p.tiles_a;
    const __half* Z = isA ? p.X : p.dY;
    const int64_t ldz = isA ? p.ldx : p.ldy, cols = isA ? p.K : p.N;
    const float* S = isA ? p.P : p.T;
    const int64_t c0 = (int64_t)(isA ? tile : tile - p.tiles_a) * kFgCols;
    const int64_t first = p.order ? __ldcg(p.start + a) : 0;
    const int64_t last = p.order ? __ldcg(p.start + a + 1) : (a == 0 ? p.M : 0);
    const int64_t chunks = (last - first + kFgTokens - 1) / kFgTokens;
    const uint32_t smem = (uint32_t)__cvta_generic_to_shared(fg_smem);

    // stage s: [64 tokens][kFgZ] fp16 columns, then [64 tokens][SS] fp32; a thread's
    // 16-byte pieces are one column of every ZR-th (SR-th) token
    constexpr int ZG = kFgCols / 8, SG = RC / 4, ZR = kFgThreads / ZG, SR = kFgThreads / SG;
    const int zr = tid / ZG, zq = tid % ZG, sr = tid / SG, sq = tid % SG;
    const bool zin = c0 + 8 * zq < cols, sin = j0 + 4 * sq < p.ld;
    const __half* zsrc = Z + c0 + 8 * zq;
    const float* ssrc = S + j0 + 4 * sq;
    const uint32_t zdst = smem + (uint32_t)(zr * kFgZ * 2 + zq * 16);
    const uint32_t sdst = smem + (uint32_t)(kFgTokens * kFgZ * 2 + sr * G::SS * 4 + sq * 16);
    const int total = (int)(last - first);
    const int32_t* list = p.order ? p.order + first : nullptr;
    auto fill = [&](int64_t c, int s) {
        if (c < chunks) {
            const uint32_t stage = (uint32_t)(s * G::STAGE);
            const int l0 = (int)c * kFgTokens;
#pragma unroll
            for (int u = 0; u < kFgTokens / ZR; ++u) {
                const int l = l0 + zr + u * ZR;
                const bool in = zin && l < total;
                const int64_t m = in ? (list ? __ldcg(list + l) : l) : 0;
                cp16(zdst + stage + (uint32_t)(u * ZR * kFgZ * 2), in ? zsrc + m * ldz : Z, in ? 16u : 0u);
            }
#pragma unroll
            for (int u = 0; u < (kFgTokens + SR - 1) / SR; ++u) {
                const int l = l0 + sr + u * SR;
                const bool in = sin && l < total;
                const int64_t m = in ? (list ? __ldcg(list + l) : l) : 0;
                if (SR <= kFgTokens || sr < kFgTokens)
                    cp16(sdst + stage + (uint32_t)(u * SR * G::SS * 4), in ? ssrc + m * p.ld : S,
                         in ? 16u : 0u);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    float sum[2][NT][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[b][n][e] = 0.0f;
    const int cols32 = (warp & 1) * 32, th = (warp >> 1) * 16;    // columns, tokens of the warp

#pragma unroll
    for (int s = 0; s < kFgStages - 1; ++s) fill(crank + (int64_t)s * csize, s);
    int it = 0;
    for (int64_t c = crank; c < chunks; c += csize, ++it) {
        fill(c + (int64_t)(kFgStages - 1) * csize, (it + kFgStages - 1) % kFgStages);
        asm volatile("cp.async.wait_group %0;" ::"n"(kFgStages - 1) : "memory");
        __syncthreads();
        const uint8_t* st = fg_smem + (it % kFgStages) * G::STAGE;
        const __half* zs = reinterpret_cast<const __half*>(st);
        const float* ss = reinterpret_cast<const float*>(st + kFgTokens * kFgZ * 2);
        float acc[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[b][n][e] = 0.0f;
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8) {
            const int r0 = th + 8 * k8 + t, r1 = r0 + 4;
            // MMA rows g and g + 8 of block b are columns 2g and 2g + 1 of its 16
            uint32_t a[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const int c = cols32 + 16 * b + 2 * g;
                const uint32_t z0 = *reinterpret_cast<const uint32_t*>(zs + r0 * kFgZ + c);
                const uint32_t z1 = *reinterpret_cast<const uint32_t*>(zs + r1 * kFgZ + c);
                a[b][0] = half_bits_f32(z0, 0);
                a[b][1] = half_bits_f32(z0, 1);
                a[b][2] = half_bits_f32(z1, 0);
                a[b][3] = half_bits_f32(z1, 1);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                uint32_t h0, l0, h1, l1;
                split_tf32(ss[r0 * G::SS + 8 * n + g], h0, l0);
                split_tf32(ss[r1 * G::SS + 8 * n + g], h1, l1);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    mma_tf32(acc[b][n], a[b][0], a[b][1], a[b][2], a[b][3], l0, l1);
                    mma_tf32(acc[b][n], a[b][0], a[b][1], a[b][2], a[b][3], h0, h1);
                }
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) sum[b][n][e] = __fadd_rn(sum[b][n][e], acc[b][n][e]);
        // (with two stages the next fill overwrites the one just read)
        __syncthreads();
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                     // the stages are free

    // the token quarters, then the cluster's parts, as [column][rank]
    constexpr int RE = kFgCols * RC;
    float* red = reinterpret_cast<float*>(fg_smem);
    float* xred = red + 4 * RE;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(warp >> 1) * RE + (cols32 + 16 * b + 2 * g + (e >> 1)) * RC + 8 * n + 2 * t + (e & 1)] =
                    sum[b][n][e];
    __syncthreads();
    auto quarters = [&](int e) {
        return __fadd_rn(__fadd_rn(red[e], red[RE + e]), __fadd_rn(red[2 * RE + e], red[3 * RE + e]));
    };
    if (csize > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (crank != 0) {
            float* dst = cg::this_cluster().map_shared_rank(xred, 0) + (crank - 1) * RE;
            for (int e = tid; e < RE; e += kFgThreads) dst[e] = quarters(e);
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    if (crank != 0) return;
    for (int i = tid; i < RE; i += kFgThreads) {
        // dA is stored [rank][column], dB [column][rank]: adjacent threads write
        // adjacent values of either
        const int col = isA ? i % kFgCols : i / RC, j = isA ? i / kFgCols : i % RC;
        const int e = col * RC + j;
        float v = quarters(e);
        for (int c = 1; c < csize; ++c) v = __fadd_rn(v, xred[(c - 1) * RE + e]);
        if (c0 + col < cols && j0 + j < p.rank) {
            if (isA) p.dA[((int64_t)a * p.rank + j0 + j) * p.K + c0 + col] = v;
            else p.dB[((int64_t)a * p.N + c0 + col) * p.rank + j0 + j] = v;
        }
    }
}

template <int NT>
cudaError_t launch_fg(const FactorGradParams& p, int tiles, cudaStream_t stream) {
    using G = FgGeo<NT>;
    auto kern = factor_grad_kernel<NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::BYTES);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t zc = (p.ld + G::RC - 1) / G::RC;
    // share out an adapter's tokens while the grid is short of two CTAs per SM and
    // each CTA keeps two stages of them
    int csize = 1;
    while (csize < kFgMaxCluster && (int64_t)tiles * p.count * zc * csize < 2 * sms &&
           p.M >= (int64_t)4 * csize * kFgTokens)
        csize *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)csize;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)(tiles * csize), (unsigned)p.count, (unsigned)zc);
    cfg.blockDim = dim3(kFgThreads);
    cfg.dynamicSmemBytes = G::BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p, csize);
}

// dY with its rows padded by zeros to a multiple of 8 values (16 bytes).
__global__ void pad_rows_kernel(const __half* __restrict__ src, int64_t M, int64_t N, int64_t ld,
                                __half* __restrict__ dst) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * ld;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / ld, n = i - m * ld;
        dst[i] = n < N ? src[m * N + n] : __float2half_rn(0.0f);
    }
}

}  // namespace

cudaError_t launch_shrink(const ShrinkParams& p, cudaStream_t stream) {
    const auto addr = reinterpret_cast<uintptr_t>(p.F);
    if (p.dtype == 0 && p.sk == 1 && (addr & 15u) == 0 && p.sj % 8 == 0 && p.sa % 8 == 0 &&
        p.K % 8 == 0)
        return launch_shrink_form<kKPairs>(p, stream);
    if (p.dtype == 0 && p.sj == 1 && (addr & 3u) == 0 && p.rank % 2 == 0 && p.sk % 2 == 0 &&
        p.sa % 2 == 0)
        return launch_shrink_form<kJPairs>(p, stream);
    if (p.dtype != 0 && p.sk == 1 && (addr & 15u) == 0 && p.sj % 8 == 0 && p.sa % 8 == 0 &&
        p.K % 8 == 0)
        return p.dtype == 1 ? launch_shrink_form<kKBf16>(p, stream)
                            : launch_shrink_form<kKF32>(p, stream);
    if (p.dtype != 0 && p.sj == 1)
        return p.dtype == 1 ? launch_shrink_form<kJBf16>(p, stream)
                            : launch_shrink_form<kJF32>(p, stream);
    return launch_shrink_form<kAnyType>(p, stream);
}

cudaError_t launch_order(const int32_t* index, int64_t M, int count, int32_t* order,
                         int32_t* start, bool beside, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)count);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, order_kernel, index, M, count, order, start);
}

cudaError_t launch_factor_grads(FactorGradParams p, cudaStream_t stream) {
    p.tiles_a = p.dA ? (int)((p.K + kFgCols - 1) / kFgCols) : 0;
    const int tiles_b = p.dB ? (int)((p.N + kFgCols - 1) / kFgCols) : 0;
    const int tiles = p.tiles_a + tiles_b;
    return p.ld <= 16 ? launch_fg<2>(p, tiles, stream)
         : p.ld <= 32 ? launch_fg<4>(p, tiles, stream)
                      : launch_fg<8>(p, tiles, stream);
}

cudaError_t launch_pad_rows(const __half* src, int64_t M, int64_t N, int64_t ld, __half* dst,
                            cudaStream_t stream) {
    const int64_t blocks = (M * ld + 1023) / 1024;
    pad_rows_kernel<<<(unsigned)(blocks < 148 * 16 ? blocks : 148 * 16), 256, 0, stream>>>(src, M, N,
                                                                                        ld, dst);
    return cudaGetLastError();
}

}  // namespace hqq
