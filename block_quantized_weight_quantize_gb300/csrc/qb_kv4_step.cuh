// qb_kv4_step.cuh -- attention of a few new tokens a sequence over the paged
// 4-bit cache (qgemv.h: kv4_attn), for a head size DP.
//
// Mathematics.  With a key's codes c and steps D, a score is
//     z = scale * sum_G D_G (sum_{e in G} q_e (c_e - 8)),
// so the tensor cores multiply queries by whole codes and the steps come in as
// one f32 factor a (key, group).  The output is
//     o_e = sum_i (p_i D_iG) (c_ie - 8) / sum_i p_i,  p_i = 2^(z_i - m),
// again a product with whole codes, of the probabilities times the steps.  m is
// the running maximum; sums and maxima are f32.
//
// Operands.  The codes are the A side (16 keys, or 16 of the value's elements, by
// 16), the rows the 8 columns of the B side, since a step has few rows: 4 rows as
// pairs (high part, low part), or 8 rows, in f32 with a product more for their low
// parts; of more rows there are more tiles, each with the keys anew.  Codes become
// f16 without a conversion: a code in the low bits of an f16 is the subnormal
// c * 2^-24, exact, and 1024 + c is one OR away.  Half-precision tiles of 8 take the
// first for keys, with -8 * sum of the queries as the sums' initial value; elsewhere
// a packed addition takes 1032 off (the sum of q or p times 8 taken off at the end
// costs f32 its last three bits: an error of 1.4e-6 against 2.1e-7).  Queries are
// scaled by a power of two a row to f16's top; in f32 they enter as two f16 (22
// bits).  The probabilities times steps likewise, scaled by a power of two a row that
// follows the largest step that the row sees (as the running maximum does; one for all
// rows of a tile would let a row's bits depend on values that it does not see), and
// pass from the scores' layout to the B side by an 8 x 8 transpose in registers.
//
// Layout.  A lane of the A fragment (row g, slots of t) needs 8 elements of key g
// in one word: the cache's key rows are ordered so that one wide load holds a
// lane's words of all groups; value rows so that it holds a lane's halves.
// Rows of 8 are keys in the order 0 7 1 6 2 5 3 4 (row 2t: key t, 2t + 1: key
// 7 - t), which keeps both loads free of bank conflicts.
//
// Work.  Units of 32 keys of one (sequence, key head, row tile), counted along
// the whole batch with 64 keys' worth more for an item's own cost; every block takes the
// same count of consecutive units whatever the sequences' lengths are, its warps
// the same count of those, and each warp streams its own through a ring of bulk copies (a page's block of a
// head is contiguous), so warps do not wait for one another until the end.  Then
// the block joins the pieces of the items that its warps share; an item that
// blocks share is joined by kv4_combine_kernel, in the order of the keys.
//
// Measured: 64 sequences of up to 8192 keys (297 MB of cache), one token each in f32,
// 32 heads of 128 on 8 key heads: 78.4 us, 3.9 TB/s.  Instructions bound it (49 million a
// call, 2.2 a cycle and multiprocessor; with the arithmetic taken out the copies alone
// took 60 us, and the arithmetic alone 69).  One sequence of 131071 keys in bf16 (151 MB):
// 48 us, 3.2 TB/s, of which some 10 are the start and 8 the joins.
#pragma once

#include <algorithm>
#include <climits>
#include <type_traits>

#include "qb_kv4.cuh"

namespace qb {

constexpr int kSeqChunk = 32;   // sequences summed together in a block's table

// Rows (token, query head) of a row tile: 4, as pairs of high and low part, or 8.
__host__ __device__ constexpr int step_rows(bool pair) { return pair ? 4 : 8; }
// Keys of a unit.  (64 where a lane's registers hold them: 256 steps on 1000 keys in
// f32, 32 heads of 128, 8 key heads 114 us against 87; one on 16000 15.6 against 16.3.)
constexpr int kUnit = 32;
// Warps of a block (one a multiprocessor), by the registers that a lane's sums
// (dp / 4) and queries take.
__host__ __device__ constexpr int step_warps(int dp) { return dp > 128 ? 8 : 12; }
__host__ __device__ constexpr int step_unit_bytes(int dp) { return kv4_block(kUnit, dp); }
// Units a warp's ring holds: what the 227 KB a block may have leave beside its tables (2072 bytes, 548 a warp, 8 a unit).
__host__ __device__ constexpr int step_stages(int dp) {
    const int w = step_warps(dp);
    const int n = (232448 - 2072 - w * 548) / (w * (step_unit_bytes(dp) + 8));
    return n > 8 ? 8 : n;
}
// Byte offsets of the workspace's parts.
struct StepWs {
    int64_t part, stat, cpart, cstat, meta, last, end;
};
inline StepWs step_ws(int64_t grid, int64_t warps, int64_t rows, int64_t dp) {
    StepWs w;
    w.part = 0;
    w.cpart = w.part + grid * warps * 2 * rows * dp * 4;
    w.stat = w.cpart + grid * 2 * rows * dp * 4;
    w.cstat = w.stat + grid * warps * 2 * rows * 8;
    w.meta = w.cstat + grid * 2 * rows * 8;
    w.last = w.meta + grid * 16;
    w.end = (w.last + grid * 4 + 15) / 16 * 16;
    return w;
}

struct StepK {
    Kv4AttnArgs a;
    int grp;          // query heads a key head
    int nosplit;      // a block's share is whole items
    int min_share;    // units a block
    float *part;      // [grid][warps][2][rows][DP]: a warp's pieces (0: of an item begun before it)
    float2 *stat;     // [grid][warps][2][rows] running maximum, sum
    float *cpart;     // [grid][2][rows][DP]: a block's pieces, joined
    float2 *cstat;
    int *last;        // [grid] the last block that holds a piece of the item that starts here and goes on; -1: none
    int4 *meta;       // [grid] that item's first token, tokens, key head, row tile
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c = a b + d
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, float d0, float d1, float d2, float d3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(d0), "f"(d1), "f"(d2), "f"(d3));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    mma_f16(c, a0, a1, a2, a3, b0, b1, c[0], c[1], c[2], c[3]);
}
// An 8 x 8 matrix of f16, a row's two neighbours a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// W words (or W halves) of shared memory in one load
template <int N>
__device__ __forceinline__ void lds(const uint8_t *p, uint32_t (&w)[N]) {
    if constexpr (N == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
}

// units of U keys of one item of the sequence: from the unit of its first seen key to its end (one at least)
template <int U>
__device__ __forceinline__ void seq_units(const SeqInfo &q, int window, int &u0, int &nu) {
    const int first = kv_first_seen(q.len - q.T, window);
    u0 = first / U;
    nu = max(1, kv_parts(q.len, U) - u0);
}

// A place in the call's work: sequence, key head, row tile, unit of the key axis.
struct StepPos {
    int s, kvh, rt, u, u_end;  // u counts from the sequence's first key
    int row, len;
};

// Sequence s: from the warp's table (those from `base` on), else from memory.
__device__ __forceinline__ SeqInfo step_seq(const StepK &p, const SeqInfo *tab, int base, int s) {
    if (s < base + 32) return tab[s - base];
    return seq_info(p.a, s, false);
}

// Enters the first sequence from x.s on that has new tokens.
template <int U>
__device__ __forceinline__ SeqInfo step_enter(const StepK &p, const SeqInfo *tab, int base, StepPos &x) {
    SeqInfo q = step_seq(p, tab, base, x.s);
    while (q.T == 0 && x.s < p.a.s.nseq) q = step_seq(p, tab, base, ++x.s);
    int nu;
    seq_units<U>(q, p.a.window, x.u, nu);
    x.u_end = x.u + nu;
    x.row = q.row;
    x.len = q.len;
    return q;
}

// The item after the one that x is in; u at its beginning.
template <int R, int U>
__device__ __forceinline__ void step_item(const StepK &p, const SeqInfo *tab, int base, StepPos &x) {
    const SeqInfo q = step_seq(p, tab, base, x.s);
    if (++x.rt == (q.T * p.grp + R - 1) / R) {
        x.rt = 0;
        if (++x.kvh == p.a.c.nkv) {
            x.kvh = 0;
            ++x.s;
        }
    }
    step_enter<U>(p, tab, base, x);
}

// A joined row: E elements a lane from el on, over the sum, to (tok, head); lane 0 its lse.
template <int E>
__device__ __forceinline__ void step_store(const StepK &p, const float (&acc)[E], int el, float sum, float m, int tok,
                                           int head, int lane) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = (int64_t)tok * p.a.out_stride + (int64_t)head * p.a.c.d + el;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (el + e >= p.a.c.d) break;
        const float y = acc[e] * inv;
        if (p.a.type == QB_T_F32) static_cast<float *>(p.a.out)[at + e] = y;
        else if (p.a.type == QB_T_F16) static_cast<__half *>(p.a.out)[at + e] = __float2half_rn(y);
        else static_cast<__nv_bfloat16 *>(p.a.out)[at + e] = __float2bfloat16_rn(y);
    }
    if (lane == 0 && p.a.lse) p.a.lse[(int64_t)tok * p.a.nh + head] = (m + log2f(sum)) * 0.6931471805599453f;
}

template <int DP, bool PAIR, bool LOW, int SB>
__global__ void __launch_bounds__(step_warps(DP) * 32, 1) kv4_step_kernel(const StepK p) {
    constexpr int kWarps = step_warps(DP), kStages = step_stages(DP);
    constexpr int U = kUnit, kBytes = step_unit_bytes(DP), NB = U / 16;
    constexpr int kItemCost = 64 / U;  // what an item costs beside its units (its queries, its output), in units
    constexpr int R = step_rows(PAIR), NH = PAIR ? 1 : 2;  // rows: of a tile, a lane's
    constexpr bool CENTRE = PAIR || LOW;
    constexpr int NG = DP / 32, W = NG < 4 ? NG : 4, NP = NG / W;         // groups, groups a plane, planes
    constexpr int kSub = kv4_block(SB, DP);                               // a sub-block of SB rows in shared memory
    constexpr int kCodes = SB * DP / 2, kSteps = SB * DP / 16, kPlane = SB * 16 * W;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bars[kWarps][kStages];
    __shared__ long long chunk_sum[8192 / kSeqChunk + 1];
    __shared__ SeqInfo tabs[kWarps][32];  // a warp's sequences, from its first one's chunk on
    __shared__ int4 piece[kWarps][2];     // a warp's pieces: first token, tokens (0: none), key head, row tile
    __shared__ int piece_ends[kWarps];    // its piece of an item begun before it ends that item
    __shared__ int failed, item_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * kStages * kBytes;
    uint64_t *full = full_bars[warp];
    // the pieces that a unit is copied in, a lane each
    const int pieces = SB < p.a.c.page ? 2 * (NP + 1) : U / SB;
    if (lane < kStages) mbar_init(full + lane, pieces);
    fence_mbar_init();
    if (lane < 2) piece[warp][lane] = make_int4(0, 0, 0, 0);
    if (threadIdx.x == 0) failed = 0;
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();

    // ---- the work.  An item's place on the line of units: kItemCost, then its own
    const int nseq = p.a.s.nseq, nchunks = (nseq + kSeqChunk - 1) / kSeqChunk;
    SeqInfo *tab = tabs[warp];
    int base = 0;
    struct Weight {
        int nu, nrt;
        long long n;
    };
    auto weight = [&](const SeqInfo &q) {
        Weight w;
        int u0;
        seq_units<U>(q, p.a.window, u0, w.nu);
        w.nrt = (q.T * p.grp + R - 1) / R;
        w.n = (long long)p.a.c.nkv * w.nrt * (w.nu + kItemCost);
        return w;
    };
    long long total;
    if (nchunks == 1) {  // every warp by itself
        const SeqInfo q = seq_info(p.a, lane, blockIdx.x == 0 && warp == 0);
        tab[lane] = q;
        total = weight(q).n;
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        __syncwarp();
    } else {
        for (int c = warp; c < nchunks; c += kWarps) {
            long long n = weight(seq_info(p.a, c * kSeqChunk + lane, blockIdx.x == 0)).n;
#pragma unroll
            for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
            if (lane == 0) chunk_sum[c] = n;
        }
        __syncthreads();
        if (warp == 0) {
            long long carry = 0;
            for (int c0 = 0; c0 < nchunks; c0 += 32) {
                const long long n = c0 + lane < nchunks ? chunk_sum[c0 + lane] : 0;
                long long sum = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                    if (lane >= o) sum += y;
                }
                if (c0 + lane < nchunks) chunk_sum[c0 + lane] = carry + sum - n;
                carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
            if (lane == 0) chunk_sum[nchunks] = carry;
        }
        __syncthreads();
        total = chunk_sum[nchunks];
    }
    long long share = (total + gridDim.x - 1) / gridDim.x;
    if (share < p.min_share) share = p.min_share;
    // Finds place x on the line: its sequence, the item in it and the place in the item.
    struct Found {
        int s, nrt, item, at;
    };
    auto find = [&](long long x) {
        long long before = 0;
        if (nchunks > 1) {
            int lo = 0, hi = nchunks;  // the chunk that holds it
            while (hi - lo > 1) {
                const int m = (lo + hi) / 2;
                if (chunk_sum[m] <= x) lo = m; else hi = m;
            }
            base = lo * kSeqChunk;
            before = chunk_sum[lo];
            const SeqInfo q = seq_info(p.a, base + lane, false);
            __syncwarp();
            tab[lane] = q;
            __syncwarp();
        }
        const Weight w = weight(tab[lane]);
        long long sum = w.n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        before += sum - w.n;
        // the last lane with units that starts at or before x
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, w.n > 0 && before <= x);
        const int l = 31 - __clz(ok);
        const long long rem = x - __shfl_sync(0xFFFFFFFFu, before, l);
        const int per = __shfl_sync(0xFFFFFFFFu, w.nu, l) + kItemCost;
        Found f;
        f.s = base + l;
        f.nrt = __shfl_sync(0xFFFFFFFFu, w.nrt, l);
        f.item = rem >> 32 ? (int)(rem / per) : (int)((uint32_t)rem / (uint32_t)per);
        f.at = (int)(rem - (long long)f.item * per);
        return f;
    };
    // the block's share; where items are not split, from an item's beginning to one
    long long b0 = min(blockIdx.x * share, total), b1 = min(b0 + share, total);
    if (p.nosplit) {
        if (b1 < total) b1 -= find(b1).at;
        if (b0 < total) b0 -= find(b0).at;
    }
    // the warp's: `count` places from x0 on
    const int wshare = (int)((b1 - b0 + kWarps - 1) / kWarps);
    const long long x0 = b0 + (long long)warp * wshare;
    int count = max(0, (int)min((long long)wshare, b1 - x0));
    StepPos cur = {};
    int place = 0;  // of the unit at `cur`, from x0 on
    if (count > 0) {
        const Found f = find(x0);
        cur.s = f.s;
        cur.kvh = f.item / f.nrt;
        cur.rt = f.item - cur.kvh * f.nrt;
        step_enter<U>(p, tab, base, cur);
        cur.u += max(0, f.at - kItemCost);
        place = max(0, kItemCost - f.at);
    }

    // ---- the copies, kStages units ahead.  A lane has one piece of a unit: a
    // page, or a part of half a page (64 tokens a page and units of 32)
    int sub_key = 0, half_mul = 0, dst_off = 0, nbytes = 0;
    const uint8_t *src = p.a.c.data;
    if (SB < p.a.c.page) {
        constexpr int kC64 = 64 * DP / 2, kS64 = 64 * DP / 16, kP64 = 64 * 16 * W;
        const int part = lane % (NP + 1), side = lane / (NP + 1);
        if (lane < 2 * (NP + 1)) {
            const bool steps = part == NP;
            nbytes = steps ? kSteps : kPlane;
            src += side * (kC64 + kS64) + (steps ? kC64 : part * kP64);
            half_mul = steps ? kS64 / 2 : kP64 / 2;
            dst_off = side * (kCodes + kSteps) + (steps ? kCodes : part * kPlane);
        }
    } else if (lane < U / SB) {
        sub_key = lane * SB;
        nbytes = kSub;
        dst_off = lane * kSub;
    }
    StepPos ahead = cur;
    int place_ahead = place;
    // page numbers of the sequence at `ahead`: lane l has the one of page pbase + l
    int pbase = 0, pcache = 0;
    auto find_pages = [&](bool fresh) {
        const int pi = (ahead.u * U) >> p.a.c.pshift;
        if (!fresh && pi + 3 < pbase + 32) return;  // a unit has four pages at most
        pbase = pi;
        pcache = 0;
        if (((int64_t)(pi + lane) << p.a.c.pshift) < ahead.len) {
            pcache = p.a.s.tables[(int64_t)ahead.row * p.a.s.maxp + pi + lane];
            if ((uint32_t)pcache >= (uint32_t)p.a.c.npages) {
                atomicOr(p.a.fault, kFaultIndex);
                pcache = 0;
            }
        }
    };
    // the next item's queries, into the cache before they are needed
    auto prefetch_queries = [&]() {
        const SeqInfo q = step_seq(p, tab, base, ahead.s);
        const int bytes = p.a.c.d * (p.a.type == QB_T_F32 ? 4 : 2), lines = (bytes + 127) / 128;
        for (int i = lane; i < R * lines; i += 32) {
            const int rho = ahead.rt * R + i / lines, j = rho / p.grp;
            if (j < q.T) {
                const int64_t at = (int64_t)(q.q0 + j) * p.a.q_stride + (int64_t)(ahead.kvh * p.grp + rho - j * p.grp) * p.a.c.d;
                asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const uint8_t *>(p.a.q) +
                                                             at * (p.a.type == QB_T_F32 ? 4 : 2) + (i % lines) * 128));
            }
        }
    };
    int islot = 0;
    auto issue = [&]() {
        if (place_ahead < count) {
            const int pg = __shfl_sync(0xFFFFFFFFu, pcache, ((ahead.u * U + sub_key) >> p.a.c.pshift) - pbase);
            if (nbytes) {  // each lane announces and issues its own piece
                if (ahead.u * U + sub_key < ahead.len) {
                    mbar_arrive_expect_tx(full + islot, (uint32_t)nbytes);
                    bulk_g2s(ring + islot * kBytes + dst_off,
                             src + ((int64_t)pg * p.a.c.nkv + ahead.kvh) * p.a.c.block_bytes +
                                 ((ahead.u & 1) ? half_mul : 0),
                             (uint32_t)nbytes, full + islot);
                } else {
                    mbar_arrive(full + islot);
                }
            }
            ++place_ahead;
            if (++ahead.u == ahead.u_end) {
                step_item<R, U>(p, tab, base, ahead);
                place_ahead += kItemCost;
                if (place_ahead < count) {
                    find_pages(true);
                    prefetch_queries();
                }
            } else {
                find_pages(false);
            }
        }
        islot = islot + 1 == kStages ? 0 : islot + 1;
    };
    if (place_ahead < count) {
        find_pages(true);
        prefetch_queries();
    }
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue();

    // ---- this lane's places in a unit
    const int krow = (g & 1) ? 7 - (g >> 1) : (g >> 1);  // the key of row g of eight
    const int koff = krow * 16 * W + t * 4 * W;
    const int voff0 = kCodes + kSteps + t * 16 * W + ((g ^ (4 * (t >> 1))) * 2 * W);
    const int voff1 = kCodes + kSteps + (7 - t) * 16 * W + ((g ^ (4 * (1 - (t >> 1)))) * 2 * W);

    const CentreK ck;
    int slot = 0;
    uint32_t phase = 0;
    while (place < count) {
        // ---- an item, or this warp's piece of it
        const int s_kvh = cur.kvh, s_rt = cur.rt, s_len = cur.len;
        const SeqInfo sq = step_seq(p, tab, base, cur.s);
        const int s_q0 = sq.q0, s_T = sq.T;
        int u0, nu;
        seq_units<U>(sq, p.a.window, u0, nu);
        const bool from_start = cur.u == u0;
        const int item_left = cur.u_end - cur.u;  // units of the item from here on
        const int units = min(item_left, count - place);
        const bool to_end = units == item_left;

        // the queries as B fragments: column g of tile n is a row (half precision) or a row's high or low part (f32)
        uint32_t B[NG][2][2];
        uint32_t BL[LOW ? NG : 1][2][2];  // the low parts
        float cinit[CENTRE ? 1 : NG][2], cs[NH];
        const int rho = s_rt * R + (PAIR ? g >> 1 : g), j = rho / p.grp;
        const bool live = j < s_T;
        const int64_t at = (int64_t)(s_q0 + j) * p.a.q_stride + (int64_t)(s_kvh * p.grp + rho - j * p.grp) * p.a.c.d;
        auto load = [&](int G, float (&x)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.0f;
            const int el = G * 32 + t * 8;
            if (!live || el >= p.a.c.d) return;
            if (LOW || (PAIR && p.a.type == QB_T_F32)) {
                load8<QB_T_F32>(static_cast<const float *>(p.a.q) + at + el, x);
            } else {
                const uint16_t *q = static_cast<const uint16_t *>(p.a.q) + at + el;
                if (p.a.type == QB_T_F16) load8<QB_T_F16>(q, x); else load8<QB_T_BF16>(q, x);
            }
        };
        float xs[NG][8], top = 0.0f;
#pragma unroll
        for (int G = 0; G < NG; ++G) load(G, xs[G]);
#pragma unroll
        for (int G = 0; G < NG; ++G)
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(xs[G][i]));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        // the row's largest magnitude into [2^14, 2^15)
        const int e = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 14;
        const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        // undone in the scores, with the codes' 2^-24 where they stand as subnormals
        const float back = p.a.scale * 1.4426950408889634f * exp2f((float)(e - 14 + (CENTRE ? 0 : 24)));
#pragma unroll
        for (int h = 0; h < NH; ++h) cs[h] = __shfl_sync(0xFFFFFFFFu, back, PAIR ? 8 * t : 8 * t + 4 * h);
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            float (&x)[8] = xs[G];
            float sum = 0.0f;
            uint32_t h2[4];
            // a pair's high part is cut to f16's 11 bits, its low part what is left
            float low[LOW ? 8 : 1];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = x[i] * f;
                const float hi = __uint_as_float(__float_as_uint(y) & 0xFFFFE000u);
                x[i] = !CENTRE ? y : (PAIR && (g & 1)) ? y - hi : hi;
                if constexpr (LOW) low[i] = y - hi;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) h2[i] = pack_f16(x[i], x[i + 4]);
            if constexpr (LOW) {
#pragma unroll
                for (int i = 0; i < 4; ++i) BL[G][i >> 1][i & 1] = pack_f16(low[i], low[i + 4]);
            }
            if constexpr (!CENTRE) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u = unpack_f16(h2[i]);
                    sum += u.x + u.y;
                }
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                sum *= -8.0f / 16777216.0f;
#pragma unroll
                for (int h = 0; h < 2; ++h) cinit[G][h] = __shfl_sync(0xFFFFFFFFu, sum, 8 * t + 4 * h);
                // as subnormals, every second code stands as 16 c * 2^-24
#pragma unroll
                for (int i = 1; i < 4; i += 2) {
                    __half2 &u = *reinterpret_cast<__half2 *>(&h2[i]);
                    u = __hmul2(u, __float2half2_rn(0.0625f));
                }
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                B[G][m][0] = h2[2 * m];
                B[G][m][1] = h2[2 * m + 1];
            }
        }
        // units whose keys every row sees need no mask
        const int pos_lo = s_len - s_T + (s_rt * R) / p.grp;
        const int pos_hi = s_len - s_T + min(s_T - 1, (s_rt * R + R - 1) / p.grp);
        const int first_hi = kv_first_seen(pos_hi, p.a.window);
        const int first_lo = kv_first_seen(pos_lo, p.a.window);

        float O[NG][2][4];
        float m[NH], l[NH];
        int eb[NH];  // biased exponent (binary16's) of the largest step that the row has seen
#pragma unroll
        for (int G = 0; G < NG; ++G)
#pragma unroll
            for (int i = 0; i < 8; ++i) O[G][i / 4][i % 4] = 0.0f;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.0f;
            eb[h] = 1;
        }

        auto unit = [&](const uint8_t *ub, int k0, auto masked) {
            // ---- scores: key krow + 16 b + 8 i, this lane's rows
            float z[NB][2][NH];
            uint32_t vs[NB][2][NG / 2];  // the values' steps of the same keys
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint8_t *kb = ub + (b * 16 / SB) * kSub;
                const int r0 = (b * 16) % SB;
                uint32_t st[2][NG / 2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lds<NG / 2>(kb + kCodes + (r0 + 8 * i + krow) * NG * 2, st[i]);
                    lds<NG / 2>(kb + 2 * kCodes + kSteps + (r0 + 8 * i + krow) * NG * 2, vs[b][i]);
#pragma unroll
                    for (int h = 0; h < NH; ++h) z[b][i][h] = 0.0f;
                }
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) {
                    uint32_t w0[W], w1[W];
                    lds<W>(kb + pl * kPlane + r0 * 16 * W + koff, w0);
                    lds<W>(kb + pl * kPlane + (r0 + 8) * 16 * W + koff, w1);
#pragma unroll
                    for (int gi = 0; gi < W; ++gi) {
                        const int G = pl * W + gi;
                        float acc[4];
                        uint32_t a[2][4];
#pragma unroll
                        for (int mm = 0; mm < 2; ++mm) {
                            const uint32_t x0 = mm ? w0[gi] >> 8 : w0[gi], x1 = mm ? w1[gi] >> 8 : w1[gi];
                            if constexpr (CENTRE) {
                                a[mm][0] = centre_lo(ck, x0);
                                a[mm][1] = centre_lo(ck, x1);
                                a[mm][2] = centre_hi(ck, x0);
                                a[mm][3] = centre_hi(ck, x1);
                            } else {
                                a[mm][0] = x0 & 0x000F000Fu;
                                a[mm][1] = x1 & 0x000F000Fu;
                                a[mm][2] = x0 & 0x00F000F0u;
                                a[mm][3] = x1 & 0x00F000F0u;
                            }
                        }
                        if constexpr (LOW) {  // the small products first: the tensor cores' sums lose bits at each step
                            mma_f16(acc, a[0][0], a[0][1], a[0][2], a[0][3], BL[G][0][0], BL[G][0][1], 0.0f, 0.0f, 0.0f, 0.0f);
                            mma_f16(acc, a[1][0], a[1][1], a[1][2], a[1][3], BL[G][1][0], BL[G][1][1]);
                            mma_f16(acc, a[0][0], a[0][1], a[0][2], a[0][3], B[G][0][0], B[G][0][1]);
                        } else {
                            const float c0 = CENTRE ? 0.0f : cinit[CENTRE ? 0 : G][0], c1 = CENTRE ? 0.0f : cinit[CENTRE ? 0 : G][1];
                            mma_f16(acc, a[0][0], a[0][1], a[0][2], a[0][3], B[G][0][0], B[G][0][1], c0, c1, c0, c1);
                        }
                        mma_f16(acc, a[1][0], a[1][1], a[1][2], a[1][3], B[G][1][0], B[G][1][1]);
                        const float2 d0 = unpack_f16(st[0][G / 2]), d1 = unpack_f16(st[1][G / 2]);
                        const float s0 = (G & 1) ? d0.y : d0.x, s1 = (G & 1) ? d1.y : d1.x;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int h = PAIR ? 0 : c;
                            z[b][0][h] = fmaf(s0, acc[c], z[b][0][h]);
                            z[b][1][h] = fmaf(s1, acc[2 + c], z[b][1][h]);
                        }
                    }
                }
            }
            uint32_t seen[NH];  // bit 2 b + i: the row sees that key
            if constexpr (masked) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    const int j = (s_rt * R + (PAIR ? t : 2 * t + h)) / p.grp;
                    const int pos = j < s_T ? s_len - s_T + j : -1;
                    const int first = kv_first_seen(pos, p.a.window);
                    seen[h] = 0;
#pragma unroll
                    for (int k = 0; k < 2 * NB; ++k) {
                        const int key = k0 + 8 * k + krow;
                        if (key >= first && key <= pos) seen[h] |= 1u << k;
                    }
                }
            }
            // ---- the running maximum and the steps' largest exponent; both rarely move
            // the keys that a row does not see, and places that hold no key, may hold any step
            auto largest_step = [&](int h) {
                __half2 top2 = __float2half2_rn(0.0f);
                auto steps = [&](int k, int i) {
                    if constexpr (masked) return seen[h] >> k & 1 ? vs[k >> 1][k & 1][i] : 0u;
                    else return vs[k >> 1][k & 1][i];
                };
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i) {
                        const uint32_t u = steps(k, i);
                        top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __half2 *>(&u)));
                    }
                top2 = __hmax2(top2, __lowhigh2highlow(top2));
                uint32_t tb = *reinterpret_cast<const uint32_t *>(&top2) & 0xFFFFu;
                if (tb >= 0x7C00u) {  // a step that is not finite says nothing about the others
                    tb = 0;
#pragma unroll
                    for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                        for (int i = 0; i < NG / 2; ++i) {
                            const uint32_t u = steps(k, i), lo = u & 0x7FFFu, hi = u >> 16 & 0x7FFFu;
                            if (lo < 0x7C00u) tb = max(tb, lo);
                            if (hi < 0x7C00u) tb = max(tb, hi);
                        }
                }
                return tb;
            };
            uint32_t tb[NH];
            tb[0] = largest_step(0);
            if constexpr (NH == 2) tb[1] = masked ? largest_step(1) : tb[0];
            bool moved = false;
            float top[NH];
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                top[h] = m[h];
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) {
                    float y = z[k >> 1][k & 1][h] * cs[h];
                    if constexpr (masked) {
                        if (!(seen[h] >> k & 1)) y = -INFINITY;
                    }
                    z[k >> 1][k & 1][h] = y;
                    top[h] = fmaxf(top[h], y);
                }
                moved |= top[h] > m[h] || (int)(tb[h] >> 10) > eb[h];
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
                float f[NH];
#pragma unroll
                for (int h = 0; h < NH; ++h) {
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) {
                        top[h] = fmaxf(top[h], __shfl_xor_sync(0xFFFFFFFFu, top[h], o));
                        tb[h] = max(tb[h], __shfl_xor_sync(0xFFFFFFFFu, tb[h], o));
                    }
                    const int eb_new = max(eb[h], (int)(tb[h] >> 10));
                    const float fe = __uint_as_float((uint32_t)(127 + eb[h] - eb_new) << 23);
                    eb[h] = eb_new;
                    f[h] = top[h] == m[h] ? 1.0f : ex2(m[h] - top[h]);
                    l[h] *= f[h];
                    f[h] *= fe;
                    m[h] = top[h];
                }
#pragma unroll
                for (int G = 0; G < NG; ++G)
#pragma unroll
                    for (int i = 0; i < 8; ++i) O[G][i / 4][i % 4] *= f[PAIR ? 0 : i & 1];
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const float pe = __uint_as_float((uint32_t)(127 + 28 - eb[h]) << 23);  // |step| * pe < 2^14
                const float mm = m[h] == -INFINITY ? 0.0f : m[h];
#pragma unroll
                for (int k = 0; k < 2 * NB; ++k) {
                    const float e = ex2(z[k >> 1][k & 1][h] - mm);
                    l[h] += e;
                    z[k >> 1][k & 1][h] = e * pe;
                }
            }

            // ---- the values' codes times probabilities times steps
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const uint8_t *va = ub + (b * 16 / SB) * kSub + ((b * 16) % SB) * 16 * W, *vb = va + 8 * 16 * W;
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) {
                    uint32_t c00[W / 2], c01[W / 2], c10[W / 2], c11[W / 2];
                    lds<W / 2>(va + pl * kPlane + voff0, c00);
                    lds<W / 2>(va + pl * kPlane + voff1, c01);
                    lds<W / 2>(vb + pl * kPlane + voff0, c10);
                    lds<W / 2>(vb + pl * kPlane + voff1, c11);
#pragma unroll
                    for (int gi = 0; gi < W; ++gi) {
                        const int G = pl * W + gi;
                        uint32_t x[2];
                        [[maybe_unused]] uint32_t xl[2];  // the low parts
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float2 d2 = unpack_f16(vs[b][i][G / 2]);
                            const float d = (G & 1) ? d2.y : d2.x;
                            float x0 = z[b][i][0] * d, x1 = PAIR ? 0.0f : z[b][i][NH - 1] * d;
                            if constexpr (masked) {  // a key that the row does not see may hold a step that is not finite
                                if (!(seen[0] >> (2 * b + i) & 1)) x0 = 0.0f;
                                if (!(seen[NH - 1] >> (2 * b + i) & 1)) x1 = 0.0f;
                            }
                            const float hi = __uint_as_float(__float_as_uint(x0) & 0xFFFFE000u);  // f16's 11 bits
                            if constexpr (PAIR) {
                                x1 = x0 - hi;
                                x0 = hi;
                            } else if constexpr (LOW) {
                                const float hi1 = __uint_as_float(__float_as_uint(x1) & 0xFFFFE000u);
                                xl[i] = transpose8(pack_f16(x0 - hi, x1 - hi1));
                                x0 = hi;
                                x1 = hi1;
                            }
                            x[i] = transpose8(pack_f16(x0, x1));
                        }
                        const uint32_t y0 = __byte_perm(c00[gi / 2], c01[gi / 2], (gi & 1) ? 0x7632 : 0x5410);
                        const uint32_t y1 = __byte_perm(c10[gi / 2], c11[gi / 2], (gi & 1) ? 0x7632 : 0x5410);
#pragma unroll
                        for (int mm = 0; mm < 2; ++mm) {
                            const uint32_t v0 = mm ? y0 >> 8 : y0, v1 = mm ? y1 >> 8 : y1;
                            const uint32_t a0 = centre_lo(ck, v0), a1 = centre_hi(ck, v0), a2 = centre_lo(ck, v1), a3 = centre_hi(ck, v1);
                            if constexpr (LOW) {  // added here, rounded: 2.4e-7 off 64 bits, 8.7e-7 as products into O, 4% faster
                                float y[4];
                                mma_f16(y, a0, a1, a2, a3, xl[0], xl[1], 0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                                for (int i = 0; i < 4; ++i) O[G][mm][i] += y[i];
                            }
                            mma_f16(O[G][mm], a0, a1, a2, a3, x[0], x[1]);
                        }
                    }
                }
            }
        };

        for (int u = cur.u; u < cur.u + units; ++u) {
            const int k0 = u * U;
            const bool landed = mbar_wait_bounded(full + slot, phase, p.a.fault);
            if (!__all_sync(0xFFFFFFFFu, landed)) {  // a copy never completed: fault word raised
                failed = 1;
                count = -1;
                cur.u = u;
                break;
            }
            const uint8_t *ub = ring + slot * kBytes;
            if (k0 > pos_hi || k0 <= first_lo - U)
                ;  // no row sees it: the sequence's other row tiles do
            else if (k0 + U - 1 > pos_lo || k0 < first_hi)
                unit(ub, k0, std::true_type());
            else
                unit(ub, k0, std::false_type());
            __syncwarp();  // every lane has read the slot
            issue();
            slot = slot + 1 == kStages ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
        }

        if (count < 0) break;

        // ---- the item's rows: out, or this piece's sums
        const bool whole = from_start && to_end;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float sum = l[h];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float fo = __uint_as_float((uint32_t)(127 - 28 + eb[h]) << 23);  // undoes pe
            const float f = !whole ? fo : sum == 0.0f ? 0.0f : fo / sum;
            const int row = (PAIR ? t : 2 * t + h), rho = s_rt * R + row, j = rho / p.grp;
            if (j >= s_T) continue;
            const int64_t tok = s_q0 + j;
            const int head = s_kvh * p.grp + rho - j * p.grp;
            const int64_t rec = (int64_t)((blockIdx.x * kWarps + warp) * 2 + (from_start ? 1 : 0)) * R + row;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                float x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float (&o)[4] = O[G][i / 2];
                    const int c = (i & 1) * 2;
                    x[i] = (PAIR ? o[c] + o[c + 1] : o[c + h]) * f;
                }
                const int el = G * 32 + g * 4;
                if (!whole) {
                    *reinterpret_cast<float4 *>(p.part + rec * DP + el) = make_float4(x[0], x[1], x[2], x[3]);
                } else if (el < p.a.c.d) {
                    const int64_t at = tok * p.a.out_stride + (int64_t)head * p.a.c.d + el;
                    if (LOW || (PAIR && p.a.type == QB_T_F32)) {
                        *reinterpret_cast<float4 *>(static_cast<float *>(p.a.out) + at) = make_float4(x[0], x[1], x[2], x[3]);
                    } else {
                        uint2 u;
                        if (p.a.type == QB_T_F16) {
                            u = make_uint2(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]));
                        } else {
                            const __nv_bfloat162 lo = __floats2bfloat162_rn(x[0], x[1]), hi = __floats2bfloat162_rn(x[2], x[3]);
                            u = make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                        }
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.a.out) + at) = u;
                    }
                }
            }
            if (g == 0) {
                if (!whole)
                    p.stat[rec] = make_float2(m[h], sum);
                else if (p.a.lse)
                    p.a.lse[tok * p.a.nh + head] = (m[h] + log2f(sum)) * 0.6931471805599453f;
            }
        }
        if (!whole && lane == 0) {
            piece[warp][from_start ? 1 : 0] = make_int4(s_q0, s_T, s_kvh, s_rt);
            if (!from_start) piece_ends[warp] = to_end;
            if (!to_end && x0 + count == b1)  // the block that holds the item's last unit
                item_last = (int)((x0 + place + item_left - 1) / share);
        }
        place += units;
        if (to_end) {
            step_item<R, U>(p, tab, base, cur);
            place += kItemCost;
        } else {
            cur.u += units;
        }
    }

    // a block does not end while copies issued after one that was given up may still write its memory (waits bounded too)
    if (count < 0) {
#pragma unroll 1
        for (int i = 1; i < kStages; ++i) {
            if (++cur.u == cur.u_end) step_item<R, U>(p, tab, base, cur);
            if (cur.u == ahead.u && cur.rt == ahead.rt && cur.kvh == ahead.kvh && cur.s == ahead.s) break;
            slot = slot + 1 == kStages ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
            mbar_wait_bounded(full + slot, phase, p.a.fault);
        }
    }

    // ---- the items that the block's warps share: a warp takes a row of one
    __syncthreads();
    if (failed) {
        if (threadIdx.x == 0) p.last[blockIdx.x] = -1;
        return;
    }
    // warps that hold the start of an item that goes on, a piece of one begun before them, one that ends it
    const bool in = lane < kWarps;
    const uint32_t starts = __ballot_sync(0xFFFFFFFFu, in && piece[in ? lane : 0][1].y != 0);
    const uint32_t goes = __ballot_sync(0xFFFFFFFFu, in && piece[in ? lane : 0][0].y != 0);
    const uint32_t ends = __ballot_sync(0xFFFFFFFFu, in && piece[in ? lane : 0][0].y != 0 && piece_ends[in ? lane : 0]);
    const int carried = goes & 1;  // the block's first item was begun by another block
    const int nshared = carried + __popc(starts);
    int goes_on = 0;  // the last item goes on in the next block
    if (starts) {
        const int w = 31 - __clz(starts);
        goes_on = (ends >> w >> 1) == 0;
    }
    for (int task = warp; task < nshared * R; task += kWarps) {
        const int k0 = task / R, row = task - k0 * R;
        const int slot_ = k0 >= carried ? 1 : 0;
        const int w = slot_ ? __fns(starts, 0, k0 - carried + 1) : 0;
        const int4 it = piece[w][slot_];
        const int rho = it.w * R + row, j = rho / p.grp;
        if (j >= it.y) continue;
        // its pieces: w's, then those of the warps after it up to the one that ends it
        const uint32_t e = slot_ ? ends >> w >> 1 : ends, g1 = goes >> w >> 1;
        const int run = __ffs(~g1) - 1;  // warps after w with a piece of an item begun before them
        const bool done = e != 0 && (slot_ ? __ffs(e) <= run : __ffs(e) - 1 <= run);
        const int parts = done ? (slot_ ? __ffs(e) + 1 : __ffs(e)) : run + 1;
        auto rec = [&](int k) { return (int64_t)((blockIdx.x * kWarps + w + k) * 2 + (k == 0 ? slot_ : 0)) * R + row; };
        constexpr int E = DP / 32;
        const float2 st = lane < parts ? p.stat[rec(lane)] : make_float2(-INFINITY, 0.0f);
        float mm = st.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
        const float wgt = ex2(st.x - (mm == -INFINITY ? 0.0f : mm));
        float sum = wgt * st.y;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        float acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = 0.0f;
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
            const float f = __shfl_sync(0xFFFFFFFFu, wgt, k);
            const float2 *x = reinterpret_cast<const float2 *>(p.part + rec(k) * DP + lane * E);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const float2 v = x[i];
                acc[2 * i] += f * v.x;
                acc[2 * i + 1] += f * v.y;
            }
        }
        if (slot_ && done) {  // wholly in this block
            step_store<E>(p, acc, lane * E, sum, mm, it.x + j, it.z * p.grp + rho - j * p.grp, lane);
        } else {
            const int64_t cr = (int64_t)(blockIdx.x * 2 + slot_) * R + row;
#pragma unroll
            for (int i = 0; i < E; ++i) p.cpart[cr * DP + lane * E + i] = acc[i];
            if (lane == 0) p.cstat[cr] = make_float2(mm, sum);
        }
    }
    if (threadIdx.x == 0) {
        p.last[blockIdx.x] = goes_on ? item_last : -1;
        if (goes_on) p.meta[blockIdx.x] = piece[31 - __clz(starts)][1];
    }
}

// Joins the pieces of items that lie in several blocks.  Every block lists the
// items (a block of the step kernel holds the start of one at most that goes on).
// A warp takes a row of one: the weights 2^(m_i - m) from the pieces' maxima, their
// sums added in the order of the keys; where there are few rows, which then have
// many pieces, a block takes a row, its warps every eighth piece.
template <int DP, int R>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const StepK p, int blocks) {
    constexpr int E = DP / 32;
    __shared__ int items[kAttnMaxGrid], lasts[kAttnMaxGrid];
    __shared__ int4 metas[kAttnMaxGrid];
    __shared__ int warp_n[8];
    __shared__ float red[8][DP], red_l[8];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mine = (int)threadIdx.x < blocks ? p.last[threadIdx.x] : -1;
    const int4 my_meta = (int)threadIdx.x < blocks ? p.meta[threadIdx.x] : make_int4(0, 0, 0, 0);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, mine >= 0);
    if (lane == 0) warp_n[warp] = __popc(b);
    __syncthreads();
    int at = __popc(b & ((1u << lane) - 1u)), nitems = 0;
    for (int w = 0; w < 8; ++w) {
        if (w < warp) at += warp_n[w];
        nitems += warp_n[w];
    }
    if (mine >= 0) {
        items[at] = threadIdx.x;
        lasts[at] = mine;
        metas[at] = my_meta;
    }
    __syncthreads();
    const int tasks = nitems * R;
    const bool wide = tasks <= 2 * (int)gridDim.x;  // a block a row
    for (int i = wide ? blockIdx.x : blockIdx.x + warp * gridDim.x; i < tasks; i += wide ? gridDim.x : 8 * gridDim.x) {
        const int c0 = items[i / R], row = i % R;
        const int4 it = metas[i / R];
        const int rho = it.w * R + row, j = rho / p.grp;
        if (j >= it.y) continue;
        const int parts = lasts[i / R] - c0 + 1;
        auto rec = [&](int k) { return (int64_t)((c0 + k) * 2 + (k == 0 ? 1 : 0)) * R + row; };
        float m = -INFINITY;
        for (int k = lane; k < parts; k += 32) m = fmaxf(m, p.cstat[rec(k)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float mm = m == -INFINITY ? 0.0f : m;
        float acc[E], l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
#pragma unroll 4
        for (int k = wide ? warp : 0; k < parts; k += wide ? 8 : 1) {
            const float2 st = p.cstat[rec(k)];
            const float wgt = ex2(st.x - mm);
            l += wgt * st.y;
            const float2 *x = reinterpret_cast<const float2 *>(p.cpart + rec(k) * DP + lane * E);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float2 v = x[e];
                acc[2 * e] += wgt * v.x;
                acc[2 * e + 1] += wgt * v.y;
            }
        }
        if (wide) {
            __syncthreads();  // red of the row before has been read
#pragma unroll
            for (int e = 0; e < E; ++e) red[warp][lane * E + e] = acc[e];
            if (lane == 0) red_l[warp] = l;
            __syncthreads();
            if (warp != 0) continue;
            l = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = 0.0f;
            for (int w = 0; w < 8; ++w) {
                l += red_l[w];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += red[w][lane * E + e];
            }
        }
        step_store<E>(p, acc, lane * E, l, m, it.x + j, it.z * p.grp + rho - j * p.grp, lane);
    }
}

// ---------------------------------------------------------------- launch

// Where the table rows hold no more keys than this, items are not split and no join
// is launched (one sequence of 100 keys: 8.3 us, 10.6 with the join, which
// a wider table takes whatever the lengths are).
constexpr int kNoSplitKeys = 256;
// A block has at least this many keys' places: on short sequences more blocks cost more in
// the join than they save, fewer leave more to each (64, 128, 256, two tokens on 200 keys in
// bf16: 12.4, 12.7, 13.3 us; one on 600: 11.9, 11.7, 12.0).
constexpr int kMinShareKeys = 128;

template <int DP, bool PAIR, bool LOW, int SB>
static int launch_step_k(StepK &p, int grid, cudaStream_t stream) {
    constexpr int kWarps = step_warps(DP), R = step_rows(PAIR);
    constexpr int smem = kWarps * step_stages(DP) * step_unit_bytes(DP);
    p.min_share = kMinShareKeys / kUnit;
    const StepWs w = step_ws(grid, kWarps, R, DP);
    p.part = reinterpret_cast<float *>(p.a.ws + w.part);
    p.stat = reinterpret_cast<float2 *>(p.a.ws + w.stat);
    p.cpart = reinterpret_cast<float *>(p.a.ws + w.cpart);
    p.cstat = reinterpret_cast<float2 *>(p.a.ws + w.cstat);
    p.last = reinterpret_cast<int *>(p.a.ws + w.last);
    p.meta = reinterpret_cast<int4 *>(p.a.ws + w.meta);
    auto *f = kv4_step_kernel<DP, PAIR, LOW, SB>;
    if (ensure_smem_limit(reinterpret_cast<const void *>(f), smem) != QB_OK) return QB_E_CUDA;
    if (const int rc = launch_pdl(f, dim3((unsigned)grid), dim3(kWarps * 32), smem, stream, p)) return rc;
    if (p.nosplit) return QB_OK;
    return launch_pdl(kv4_combine_kernel<DP, R>, dim3((unsigned)grid), dim3(256), 0, stream, p, grid);
}

template <int DP>
int launch_kv4_step(const Kv4AttnArgs &a, cudaStream_t stream) {
    StepK p = {};
    p.a = a;
    p.grp = a.nh / a.c.nkv;
    const int grid = attn_grid();
    p.nosplit = (int64_t)a.s.maxp * a.c.page <= kNoSplitKeys;
    // f32 enters as high and low parts for its accuracy: side by side in tiles of 4 rows, or in
    // tiles of 8 with a product more for the low parts, which decode a key for twice the rows.
    // By the rows a sequence and key head, on average (us in tiles of 4, of 8): 256 sequences of
    // 1000 keys, 4 rows 87, 120, half of them 4 and half 8 119, 125, 8 rows 150, 127, 16 rows 281,
    // 223, 64 rows 1023, 741; one of 600 keys, 8 rows 11.2, 13.6, 64 rows 13.9, 15.4.  Half precision
    // takes tiles of 4 where a tile of 8 would only be padded (4 rows: 88, 95), and eights from
    // there on (8 rows: 152, 102).  (Two such column tiles, which decode a key once for both, leave
    // 8 warps a multiprocessor instead of 12: up to 16 rows 182 us against 130 in bf16, 184 against
    // 180 in f32.)
    const bool low = a.type == QB_T_F32, few = a.ntok * p.grp <= (low ? 8 : 4) * (int64_t)a.s.nseq;
    if (a.c.page == 16)
        return few ? launch_step_k<DP, true, false, 16>(p, grid, stream)
               : low ? launch_step_k<DP, false, true, 16>(p, grid, stream) : launch_step_k<DP, false, false, 16>(p, grid, stream);
    return few ? launch_step_k<DP, true, false, 32>(p, grid, stream)
           : low ? launch_step_k<DP, false, true, 32>(p, grid, stream) : launch_step_k<DP, false, false, 32>(p, grid, stream);
}

}  // namespace qb
