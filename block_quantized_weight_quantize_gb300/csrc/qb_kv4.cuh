// qb_kv4.cuh -- the stored form of the paged 4-bit key/value cache (declared
// in qgemv.h) as the kernels see it: sizes, the places of codes and steps, and
// element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qb_common.cuh"
#include "qb_kv_index.h"
#include "qb_launch.h"

namespace qb {

__host__ __device__ constexpr int kv4_padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
// bytes of one (page, key head) block of `page` rows
__host__ __device__ constexpr int kv4_block(int page, int dp) { return 2 * page * (dp / 2 + dp / 16); }

struct Kv4View {
    uint8_t *data;
    int npages, page, pshift, nkv, d, dp;
    int64_t block_bytes;
};

inline Kv4View kv4_view(const qb_kv4 &c) {
    Kv4View v;
    v.data = static_cast<uint8_t *>(c.data);
    v.npages = c.npages;
    v.page = c.page;
    v.pshift = c.page == 16 ? 4 : c.page == 32 ? 5 : 6;
    v.nkv = c.nkv;
    v.d = c.d;
    v.dp = kv4_padded(c.d);
    v.block_bytes = kv4_block(c.page, v.dp);
    return v;
}

// Eight half-precision elements of `type` as f32.
template <int TYPE>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == QB_T_F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}

// Eight consecutive elements of `type` as f32; p is aligned to their size (16 or 32 bytes).
template <int TYPE>
__device__ __forceinline__ void load8(const void *p, float (&x)[8]) {
    if constexpr (TYPE == QB_T_F32) {
        const float4 a = static_cast<const float4 *>(p)[0], b = static_cast<const float4 *>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        unpack8<TYPE>(*static_cast<const uint4 *>(p), x);
    }
}

// Eight f32 values rounded once to `type` and stored.
template <int TYPE>
__device__ __forceinline__ void store8(void *p, const float (&x)[8]) {
    if constexpr (TYPE == QB_T_F32) {
        static_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        static_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == QB_T_F16) {
                const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Codes in the low (or second) four bits of each half, as code - 8.  The three
// constants stay in registers (opaque to the compiler), so that mask and OR are
// one three-input operation.
struct CentreK {
    uint32_t lo, hi, one;
    __device__ __forceinline__ CentreK() {
        asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(lo));
        asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(hi));
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(one));  // 1024, twice
    }
};
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t centre_lo(const CentreK &k, uint32_t w) {
    uint32_t b = and_or(w, k.lo, k.one);  // 1024 + c
    __half2 &h = *reinterpret_cast<__half2 *>(&b);
    h = __hadd2(h, __float2half2_rn(-1032.0f));
    return b;
}
__device__ __forceinline__ uint32_t centre_hi(const CentreK &k, uint32_t w) {
    uint32_t b = and_or(w, k.hi, k.one);  // 1024 + 16 c
    __half2 &h = *reinterpret_cast<__half2 *>(&b);
    h = __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));
    return b;
}

// Two f32 operations in one.
__device__ __forceinline__ uint64_t pair_f32(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair_f32(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__host__ __device__ constexpr int type_bytes(int type) { return type == QB_T_F32 ? 4 : 2; }

// Launchers; arguments checked by the C entries (qb_kv4_api.cu).
int launch_kv4_append(const Kv4View &c, int type, const void *k, int64_t ks, const void *v, int64_t vs,
                      const int32_t *slots, int64_t n, cudaStream_t stream);
int launch_kv4_read(const Kv4View &c, int type, const int32_t *slots, int64_t n, void *k, int64_t ks, void *v,
                    int64_t vs, cudaStream_t stream);

struct Kv4AttnArgs {
    Kv4View c;
    qb_kv_seqs s;
    int type;
    const void *q;
    int64_t q_stride;
    int64_t ntok;
    int nh;
    float scale;
    int window;
    int sinks;              // first keys that stay visible; 0 without a window
    const uint32_t *masks;  // [ntok][words] drafts that a token sees; NULL: all up to itself
    int words;
    void *out;
    int64_t out_stride;
    float *lse;
    uint8_t *ws;
    int *fault;
};
// Whether a call takes the kernels that look keys up one by one (trees, sinks).
inline bool kv4_attn_ext(const Kv4AttnArgs &a) { return a.masks != nullptr || a.sinks > 0; }
// What token j (a row's; j < T) of a sequence sees (qb_kv_index.h), and whether it sees one of the keys k0..k0+31.
__device__ __forceinline__ KvSight kv4_sight(const Kv4AttnArgs &a, int len, int T, int q0, int j) {
    const int base = len - T;
    if (a.masks) return kv_tree_sight(a.masks + (int64_t)(q0 + j) * a.words, a.words, T, base, a.window);
    return KvSight{kv_first_seen(base + j, a.window), base + j, kKvNoKey};
}
__device__ __forceinline__ uint32_t kv4_seen(const Kv4AttnArgs &a, const KvSight &s, int len, int T, int q0, int j, int k0) {
    return kv_seen_word(s, a.sinks, a.masks ? a.masks + (int64_t)(q0 + j) * a.words : nullptr, a.words, len - T, len, k0);
}
// The first key that any token from j_lo on sees beside the sinks, at the least; one that each up to j_hi sees from
// on, at the most; the last key that each from j_lo on sees before any draft or key that some do not.
__device__ __forceinline__ int kv4_first_lo(const Kv4AttnArgs &a, int len, int T, int j_lo) {
    return kv_first_seen(len - T + (a.masks ? -1 : j_lo), a.window);
}
__device__ __forceinline__ int kv4_first_hi(const Kv4AttnArgs &a, int len, int T, int j_hi) {
    return kv_first_seen(a.masks ? len - 1 : len - T + j_hi, a.window);
}
__device__ __forceinline__ int kv4_pos_lo(const Kv4AttnArgs &a, int len, int T, int j_lo) {
    return len - T + (a.masks ? -1 : j_lo);
}
__device__ __forceinline__ int kv4_pos_hi(const Kv4AttnArgs &a, int len, int T, int j_hi) {
    return a.masks ? len - 1 : len - T + j_hi;
}
// A sequence of the call: its table row, length, new tokens and first new token.
struct SeqInfo {
    int row, len, T, q0;
};
__device__ __forceinline__ SeqInfo seq_info(const Kv4AttnArgs &a, int s, bool report) {
    SeqInfo r = {0, 0, 0, 0};
    if (s >= a.s.nseq) return r;
    r.row = a.s.rows ? a.s.rows[s] : s;
    int64_t q0 = s, q1 = s + 1;
    if (a.s.q_start) {
        q0 = a.s.q_start[s];
        q1 = a.s.q_start[s + 1];
    }
    q0 = min(max(q0, (int64_t)0), a.ntok);
    q1 = min(max(q1, q0), a.ntok);
    r.q0 = (int)q0;
    r.T = (int)(q1 - q0);
    if (r.row < 0 || r.row >= a.s.nrows) {
        if (report) atomicOr(a.fault, kFaultIndex);
        r.row = 0;
    } else {
        r.len = (int)min((int64_t)max(a.s.lens[r.row], 0), (int64_t)a.s.maxp * a.c.page);
    }
    return r;
}

// Blocks of the attention kernels: one a multiprocessor.
constexpr int kAttnMaxGrid = 256;
inline int attn_grid() { return num_sms() < kAttnMaxGrid ? num_sms() : kAttnMaxGrid; }

int64_t kv4_attn_ws(int dp);
int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream);
// A few tokens a sequence (qb_kv4_step.cuh), many (qb_kv4_prompt.cuh); by padded head size.
int launch_kv4_step_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_128(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_256(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_128(const Kv4AttnArgs &a, cudaStream_t stream);
// The same for calls with trees or sinks.
int launch_kv4_step_ext_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_ext_128(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_ext_256(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_ext_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_ext_128(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_split_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_prompt_split_128(const Kv4AttnArgs &a, cudaStream_t stream);

int launch_kv_tree_masks(const int32_t *parents, int64_t ntok, const int32_t *q_start, int nseq, uint32_t *masks, int words,
                         int32_t *depth, cudaStream_t stream);
int launch_kv_tree_accept(const int32_t *parents, const int32_t *tokens, const int32_t *targets, int64_t ntok,
                          const int32_t *q_start, int nseq, int32_t *keep, int32_t *nkeep, int32_t *next, cudaStream_t stream);
int launch_kv4_keep(const qb_kv_pages &p, void *data, int nlayers, int nkv, int d, const int32_t *rows, const int32_t *q_start,
                    const int32_t *keep, const int32_t *nkeep, int64_t ntok, int n, int32_t *status, cudaStream_t stream);

int64_t kv_pages_ws(int npages, int nrows);
int launch_kv_pages_reset(const qb_kv_pages &p, cudaStream_t stream);
int launch_kv_pages_extend(const qb_kv_pages &p, const int32_t *rows, const int32_t *counts, int n, int32_t *slots,
                           int64_t nslots, int32_t *status, cudaStream_t stream);
int launch_kv_pages_fork(const qb_kv_pages &p, void *data, int nlayers, int64_t page_bytes, const int32_t *parents,
                         const int32_t *children, int n, int32_t *status, void *ws, cudaStream_t stream);
int launch_kv_pages_free(const qb_kv_pages &p, const int32_t *rows, int n, cudaStream_t stream);
int launch_kv_pages_compact(const qb_kv_pages &p, void *data, int nlayers, int64_t page_bytes, void *ws,
                            cudaStream_t stream);
int launch_kv_pages_copy(void *data, int nlayers, int64_t npages, int64_t page_bytes, const int32_t *src,
                         const int32_t *dst, int n, cudaStream_t stream);

}  // namespace qb
