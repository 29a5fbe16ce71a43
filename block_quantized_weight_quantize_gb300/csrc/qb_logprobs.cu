// qb_logprobs.cu -- log probabilities of given tokens, entropy and the largest alternatives of rows of
// logits (qgemv.h: q_logprobs).
//
// Mathematics.  With z = scale * x, X a row's largest logit and, over the row,
//     S = sum 2^d, T = sum d 2^d,  d = (x - X) * scale * log2(e),
// lse = scale X + ln S, log p(x) = scale (x - X) - ln S, and the entropy is ln S - ln(2) T / S: one pass
// gives all of it.  A thread's d is relative to a reference of its own that follows its largest element
// when that is more than 2^kLazy above it, so that a rescaling is rare; differences of
// logits are formed before they are scaled, so that rows of the type's lowest values have the
// uniform distribution that they stand for.
//
// Alternatives.  A thread remembers its largest logit and where it lies.  The j-th largest of
// these in a warp, j = ceil(k / warps), the least of the warps': at least k elements are as
// large, few are larger, and only threads whose largest reaches it can hold one.  So the row's candidates are found
// by reading those threads' elements once more (from L2), and ordered by counting.
//
// Work: a row is read by a cluster of 1 to 16 blocks, which join their sums and candidates in
// the first one's shared memory: no workspace, one launch.
#include <algorithm>
#include <cmath>
#include <cooperative_groups.h>
#include <cstdint>

#include "qb_kv4.cuh"

namespace qb {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 256, kLpWarps = kLpThreads / 32;
constexpr int kLpMaxK = QB_MAX_ALTERNATIVES, kLpMaxCluster = 16;
constexpr int kLpCand = 2048;    // candidates a block holds
constexpr float kLpLazy = 32.0f; // 2^32 times 2^24 elements stay far below f32's top

struct LpK {
    const void *x;
    int64_t stride, n;
    int vocab;
    float scale;
    const int32_t *tokens;
    int m;
    float *logp, *entropy, *lse;
    int k;
    int32_t *top_tok;
    float *top_logp;
    int cluster;
};

__device__ __forceinline__ float lp_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A logit and its place as one number: by the logit, then the lower place first.  No NaN.
__device__ __forceinline__ uint64_t lp_key(float x, uint32_t at) {
    const uint32_t b = __float_as_uint(x + 0.0f);  // -0 as +0
    return (uint64_t)(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xFFFFFFFFu - at);
}
__device__ __forceinline__ float lp_key_value(uint64_t key) {
    const uint32_t b = (uint32_t)(key >> 32);
    return __uint_as_float(b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

template <int TYPE>
constexpr int lp_vec() { return TYPE == QB_T_F32 ? 4 : 8; }

template <int TYPE>
__device__ __forceinline__ void lp_unpack(const uint4 &u, float (&x)[lp_vec<TYPE>()]) {
    if constexpr (TYPE == QB_T_F32) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    } else {
        unpack8<TYPE>(u, x);
    }
}
template <int TYPE>
__device__ __forceinline__ float lp_load(const void *row, int64_t i) {
    if constexpr (TYPE == QB_T_F32) return static_cast<const float *>(row)[i];
    else if constexpr (TYPE == QB_T_F16) return __half2float(static_cast<const __half *>(row)[i]);
    else return __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i]);
}

struct LpSums {
    float X, S, T;
    int bad;  // a NaN or +infinity
};
__device__ __forceinline__ LpSums lp_join(const LpSums &a, const LpSums &b, float s2) {
    LpSums r;
    r.X = fmaxf(a.X, b.X);
    r.bad = a.bad | b.bad;
    const float da = a.S > 0.0f ? fmaxf((a.X - r.X) * s2, -1e4f) : 0.0f, db = b.S > 0.0f ? fmaxf((b.X - r.X) * s2, -1e4f) : 0.0f;
    const float fa = lp_ex2(da), fb = lp_ex2(db);
    r.S = a.S * fa + b.S * fb;
    r.T = (a.T + a.S * da) * fa + (b.T + b.S * db) * fb;
    return r;
}

struct LpSmem {
    uint64_t cand[kLpCand];
    uint64_t joined[kLpMaxCluster * kLpMaxK];  // of the first block: every block's largest
    LpSums sums[kLpMaxCluster];
    LpSums warp_sums[kLpWarps];
    uint64_t warp_key[kLpWarps];
    uint64_t thread_key[kLpThreads];
    int count;
};

// The j-th largest of the lanes' keys (zero where fewer lanes have one).
__device__ __forceinline__ uint64_t lp_warp_nth(uint64_t key, int j) {
    uint64_t top = 0;
    for (int i = 0; i < j; ++i) {
        const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32));
        const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, (uint32_t)(key >> 32) == hi ? (uint32_t)key : 0u);
        top = (uint64_t)hi << 32 | lo;
        if (key == top) key = 0;
    }
    return top;
}

// Thins `list` (keys all different) out to few more than its k largest, then writes these in order to `out`.  By the whole block.
__device__ __forceinline__ void lp_select(LpSmem &sm, uint64_t *list, int count, int k, uint64_t *out) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int turn = 0; turn < 3 && count > kLpThreads; ++turn) {
        uint64_t mine[kLpCand / kLpThreads], top = 0;
#pragma unroll
        for (int i = 0; i < kLpCand / kLpThreads; ++i) {
            mine[i] = tid + i * kLpThreads < count ? list[tid + i * kLpThreads] : 0;
            top = max(top, mine[i]);
        }
        const uint64_t nth = lp_warp_nth(top, (k + kLpWarps - 1) / kLpWarps);
        if (lane == 0) sm.warp_key[warp] = nth;
        __syncthreads();  // the list has been read
        if (tid == 0) sm.count = 0;
        uint64_t bound = sm.warp_key[0];
        for (int w = 1; w < kLpWarps; ++w) bound = min(bound, sm.warp_key[w]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLpCand / kLpThreads; ++i)
            if (mine[i] >= bound && mine[i] != 0) list[atomicAdd(&sm.count, 1)] = mine[i];
        __syncthreads();
        count = sm.count;
        __syncthreads();
    }
    for (int i = tid; i < count; i += kLpThreads) {
        const uint64_t key = list[i];
        int rank = 0;
        for (int o = 0; o < count; ++o) rank += list[o] > key;
        if (rank < k) out[rank] = key;
    }
}

// A row as chunks of 16 bytes on their own boundaries.  The first may begin before it and the last end
// after it: these two are read element by element.
template <int TYPE>
struct LpRow {
    static constexpr int V = lp_vec<TYPE>(), ES = type_bytes(TYPE);
    const uint8_t *row;
    int lead, vocab, nchunks;  // elements of chunk 0 before the row
    int i0, i1;                // chunks that lie in the row whole
    __device__ __forceinline__ LpRow(const void *x, int vocab_) : row(static_cast<const uint8_t *>(x)), vocab(vocab_) {
        lead = (int)(reinterpret_cast<uintptr_t>(row) & 15) / ES;
        nchunks = (lead + vocab + V - 1) / V;
        i0 = lead > 0;
        i1 = (lead + vocab) / V;
    }
    __device__ __forceinline__ bool whole(int c) const { return c >= i0 && c < i1; }
    __device__ __forceinline__ int at(int c) const { return c * V - lead; }  // chunk c's first element
    __device__ __forceinline__ uint4 chunk(int c) const {
        return __ldg(reinterpret_cast<const uint4 *>(row + (int64_t)at(c) * ES));
    }
    __device__ __forceinline__ void edge(int c, float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = at(c) + i;
            x[i] = e >= 0 && e < vocab ? lp_load<TYPE>(row, e) : -INFINITY;
        }
    }
    __device__ __forceinline__ void load(int c, float (&x)[V]) const {
        if (whole(c)) lp_unpack<TYPE>(chunk(c), x);
        else edge(c, x);
    }
    // element i of chunk c as a key; zero outside the row and for what has no place in the order
    __device__ __forceinline__ uint64_t key(int c, int i, float x) const {
        const int e = at(c) + i;
        return e < 0 || e >= vocab || !(x < INFINITY) ? 0 : lp_key(x, (uint32_t)e);
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kLpThreads, 4) logprobs_kernel(const LpK p) {
    constexpr int V = lp_vec<TYPE>();
    constexpr int kAhead = 4;  // loads under way a thread
    __shared__ LpSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = p.cluster > 1 ? (int)(blockIdx.x % p.cluster) : 0;
    const int64_t row_i = blockIdx.x / p.cluster;
    pdl_launch_dependents();
    pdl_wait();
    if (p.cluster > 1) cg::this_cluster().barrier_arrive();
    const LpRow<TYPE> row(static_cast<const uint8_t *>(p.x) + row_i * p.stride * type_bytes(TYPE), p.vocab);
    const int nchunks = row.nchunks;
    const int c0 = (int)((int64_t)nchunks * rank / p.cluster), c1 = (int)((int64_t)nchunks * (rank + 1) / p.cluster);
    const float s2 = p.scale * 1.4426950408889634f;
    const float lazy = kLpLazy / s2;

    // ---- one pass
    LpSums a = {-INFINITY, 0.0f, 0.0f, 0};
    float top = __uint_as_float(0x7FC00000u);  // the thread's largest; NaN: none yet
    int top_at = -1;                           // the chunk that holds it
    auto take = [&](const uint4 &u, int c) {
        float x[V];
        lp_unpack<TYPE>(u, x);
        if (!row.whole(c)) row.edge(c, x);
        float most = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(x[i]));
        if (!(most <= top)) {
            if (!(most < INFINITY)) a.bad = 1;  // a NaN or +infinity
            else {
                top = most;
                top_at = c;
                if (most > a.X + lazy) {
                    const float d = a.S > 0.0f ? fmaxf((a.X - most) * s2, -1e4f) : 0.0f, f = lp_ex2(d);
                    a.T = (a.T + a.S * d) * f;
                    a.S *= f;
                    a.X = most;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float d = fmaxf((x[i] - a.X) * s2, -200.0f);  // 0 from -126 on
            const float e = lp_ex2(d);
            a.S += e;
            a.T += e * d;
        }
    };
    int c = c0 + tid;
    for (; c + (kAhead - 1) * kLpThreads < c1; c += kAhead * kLpThreads) {
        uint4 u[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) u[i] = row.whole(c + i * kLpThreads) ? row.chunk(c + i * kLpThreads) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) take(u[i], c + i * kLpThreads);
    }
    for (; c < c1; c += kLpThreads) take(row.whole(c) ? row.chunk(c) : make_uint4(0u, 0u, 0u, 0u), c);

    // ---- the block's sums
    if (top_at >= 0 && a.X != top) a = lp_join(a, LpSums{top, 0.0f, 0.0f, 0}, s2);
#pragma unroll
    for (int o = 16; o; o >>= 1)
        a = lp_join(a, LpSums{__shfl_xor_sync(0xFFFFFFFFu, a.X, o), __shfl_xor_sync(0xFFFFFFFFu, a.S, o),
                              __shfl_xor_sync(0xFFFFFFFFu, a.T, o), (int)__shfl_xor_sync(0xFFFFFFFFu, a.bad, o)}, s2);
    if (lane == 0) sm.warp_sums[warp] = a;
    // a lower bound of the block's k-th largest: the thread's largest, as if it were its chunk's last element
    const uint64_t mine = top_at < 0 ? 0 : lp_key(top, (uint32_t)(row.at(top_at) + V - 1));
    if (p.k) {
        sm.thread_key[tid] = mine;
        const int full = min(kLpWarps, (c1 - c0) / 32);  // warps whose threads all have elements
        const uint64_t nth = full ? lp_warp_nth(mine, (p.k + full - 1) / max(full, 1)) : 0;
        if (lane == 0) sm.warp_key[warp] = warp < full ? nth : ~uint64_t(0);
        if (tid == 0) sm.count = 0;
    }
    __syncthreads();
    if (tid == 0) {
        LpSums b = sm.warp_sums[0];
        for (int w = 1; w < kLpWarps; ++w) b = lp_join(b, sm.warp_sums[w], s2);
        sm.warp_sums[0] = b;
    }
    if (p.k) {
        uint64_t bound = sm.warp_key[0];
        for (int w = 1; w < kLpWarps; ++w) bound = min(bound, sm.warp_key[w]);
        if (bound == ~uint64_t(0)) bound = 0;
        // ---- the candidates: a warp reads the elements of a thread that may hold some
        const int per = (c1 - c0 + kLpThreads - 1) / kLpThreads;
        for (int t = warp; t < kLpThreads; t += kLpWarps) {
            // its largest may be its chunk's first element
            if (sm.thread_key[t] + (V - 1) < bound || sm.thread_key[t] == 0) continue;
            for (int i = lane; i < per; i += 32) {
                const int ch = c0 + t + i * kLpThreads;
                if (ch >= c1) break;
                float x[V];
                row.load(ch, x);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const uint64_t key = row.key(ch, e, x[e]);
                    if (key < bound || key == 0) continue;
                    const int to = atomicAdd(&sm.count, 1);
                    if (to < kLpCand) sm.cand[to] = key;
                }
            }
        }
    }
    __syncthreads();
    LpSmem *first = &sm;
    if (p.cluster > 1) cg::this_cluster().barrier_wait();  // every block has begun
    if (p.cluster > 1) first = cg::this_cluster().map_shared_rank(&sm, 0);
    if (tid == 0) first->sums[rank] = sm.warp_sums[0];
    if (p.k) {
        const int found = sm.count;
        __syncthreads();
        uint64_t *out = first->joined + rank * p.k;
        for (int i = tid; i < p.k; i += kLpThreads)
            if (i >= found) out[i] = 0;  // fewer elements than that
        if (found <= kLpCand) {
            lp_select(sm, sm.cand, found, p.k, out);
        } else {
            // more elements than fit reach the bound (long runs of rising logits): one largest after the other
            uint64_t last = ~uint64_t(0);
            for (int r = 0; r < p.k; ++r) {
                uint64_t best = 0;
                for (int ch = c0 + tid; ch < c1; ch += kLpThreads) {
                    float x[V];
                    row.load(ch, x);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const uint64_t key = row.key(ch, e, x[e]);
                        if (key < last) best = max(best, key);
                    }
                }
                best = lp_warp_nth(best, 1);
                if (lane == 0) sm.warp_key[warp] = best;
                __syncthreads();
                for (int w = 0; w < kLpWarps; ++w) best = max(best, sm.warp_key[w]);
                __syncthreads();
                if (tid == 0) out[r] = best;
                last = best;
            }
        }
    }
    if (p.cluster > 1) {
        cg::this_cluster().sync();
        if (rank != 0) return;
    } else {
        __syncthreads();
    }

    // ---- the row's, in its first block
    LpSums r = sm.sums[0];
    for (int w = 1; w < p.cluster; ++w) r = lp_join(r, sm.sums[w], s2);
    const float nan = __uint_as_float(0x7FC00000u);
    const float ln = logf(r.S);
    // (x - X) first: exact where the two are near
    auto logp = [&](float x) { return r.bad ? nan : r.S > 0.0f ? (x - r.X) * p.scale - ln : -INFINITY; };
    if (tid == 0) {
        if (p.lse) p.lse[row_i] = r.bad ? nan : r.S > 0.0f ? r.X * p.scale + ln : -INFINITY;
        if (p.entropy) p.entropy[row_i] = r.bad ? nan : r.S > 0.0f ? fmaxf(ln - 0.6931471805599453f * (r.T / r.S), 0.0f) : 0.0f;
    }
    for (int i = tid; i < p.m; i += kLpThreads) {
        const int t = p.tokens[row_i * p.m + i];
        p.logp[row_i * p.m + i] = t < 0 || t >= p.vocab ? (r.bad ? nan : -INFINITY) : logp(lp_load<TYPE>(row.row, t));
    }
    if (p.k) {
        uint64_t *best = sm.joined;
        if (p.cluster > 1) {
            best = sm.cand;
            const int all = p.cluster * p.k;
            if (all > kLpThreads) {
                lp_select(sm, sm.joined, all, p.k, best);
            } else {
                for (int i = tid; i < all; i += kLpThreads) {
                    const uint64_t key = sm.joined[i];
                    int above = 0;
                    for (int o = 0; o < all; ++o) above += sm.joined[o] > key;
                    if (key && above < p.k) best[above] = key;
                }
            }
            __syncthreads();
        }
        for (int i = tid; i < p.k; i += kLpThreads) {
            const uint64_t key = best[i];
            if (p.top_tok) p.top_tok[row_i * p.k + i] = r.bad ? -1 : (int)(0xFFFFFFFFu - (uint32_t)key);
            if (p.top_logp) p.top_logp[row_i * p.k + i] = logp(lp_key_value(key));
        }
    }
}

int launch_q_logprobs(int type, const void *x, int64_t stride, int64_t n, int vocab, float scale, const int32_t *tokens, int m,
                      float *logp, float *entropy, float *lse, int k, int32_t *top_tok, float *top_logp, cudaStream_t stream) {
    LpK p = {x, stride, n, vocab, scale, tokens, m, logp, entropy, lse, k, top_tok, top_logp, 1};
    // a cluster a row where there are few rows: two blocks a multiprocessor, each at least 2048 elements
    while (p.cluster < kLpMaxCluster && n * p.cluster < 2 * num_sms() && vocab / (2 * p.cluster) >= 2048) p.cluster *= 2;
    auto *f = type == QB_T_F32 ? logprobs_kernel<QB_T_F32> : type == QB_T_F16 ? logprobs_kernel<QB_T_F16> : logprobs_kernel<QB_T_BF16>;
    if (p.cluster > 8 && cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return QB_E_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(n * p.cluster));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, f, p) == cudaSuccess ? QB_OK : QB_E_CUDA;
}

}  // namespace qb

using namespace qb;

extern "C" int q_logprobs(qb_type type, const void *logits, int64_t row_stride, int64_t n, int64_t vocab, float scale,
                          const int32_t *tokens, int ngiven, float *logprobs, float *entropy, float *lse, int k,
                          int32_t *top_tokens, float *top_logprobs, void *stream) {
    const auto off = [](const void *p, uintptr_t b) { return (reinterpret_cast<uintptr_t>(p) & (b - 1)) != 0; };
    if (type != QB_T_F32 && type != QB_T_F16 && type != QB_T_BF16) return QB_E_ARG;
    if (n < 0 || n > (int64_t(1) << 26) || vocab < 1 || vocab > (int64_t(1) << 24) || !(scale >= 0x1p-20f && scale <= 0x1p20f) ||
        ngiven < 0 || ngiven > QB_MAX_GIVEN || k < 0 || k > QB_MAX_ALTERNATIVES || k > vocab)
        return QB_E_ARG;
    if (n == 0) return QB_OK;
    if (!logits || off(logits, type_bytes(type)) || row_stride < vocab || row_stride > (int64_t(1) << 40)) return QB_E_ARG;
    if ((ngiven > 0 && (!tokens || !logprobs)) || off(tokens, 4) || off(logprobs, 4) || off(entropy, 4) || off(lse, 4) ||
        off(top_tokens, 4) || off(top_logprobs, 4))
        return QB_E_ARG;
    return launch_q_logprobs(type, logits, row_stride, n, (int)vocab, scale, tokens, ngiven, logprobs, entropy, lse,
                             top_tokens || top_logprobs ? k : 0, top_tokens, top_logprobs, static_cast<cudaStream_t>(stream));
}
