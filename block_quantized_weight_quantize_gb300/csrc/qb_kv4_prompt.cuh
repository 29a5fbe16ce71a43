// qb_kv4_prompt.cuh -- attention of many new tokens a sequence (prompts and
// their chunks) over the paged 4-bit cache, in half precision, on the
// fifth-generation tensor cores.
//
// Mathematics: as in qb_kv4_step.cuh, but with some 100 rows and more a key head the
// products bound it, so keys and values are decoded once a tile to f16
// ((code - 8) * step, rounded once) and the tensor cores do the rest:
//     S = Q K^T (f32), P = 2^(S cs - m) (f16), O += P V (f32),
// m 11 below a running maximum, which moves only when P would pass f16's top, when
// O is rescaled in tensor memory; sums in f32.  The largest probability then lies at
// 2^11 to 2^15.9, and f16's last place, 2^-24, is 2^-35 of it or less: what is below
// 2^-36 vanishes.  m moves by whole numbers, so that a rescaled P is not rounded
// anew.  (13 instead of 11: m moves more often, 330 us for 2048 tokens on 8192 keys,
// 32 heads of 128, against 253; m at the maximum and 8 let pass: 256 us, but what is
// below 2^-25 vanishes.)
//
// A rounded key moves a score by 2^-12 of its terms, which averages out over many
// keys but not over few: lse is off by 1e-5 to 2e-5 of itself at 100 keys, 3e-6 at
// 500, 7e-7 at 2400, 3e-7 at 8192.  Where a row of an item sees fewer than kPromptFine
// keys, what the rounding leaves is decoded too (one multiply-add, exact) and multiplied
// by Q into the same scores: 1e-7 then.  It costs 10 to 46% (a prompt of 2048 tokens by
// itself, 32 heads of 128: 88 -> 97 us; 64 sequences of 64 tokens on 2000 keys: 193 ->
// 256; 2048 tokens on 8192 keys, were they to take it, 251 -> 366).  A row that sees
// more keys but weighs few of them averages nothing out: with scores of magnitudes up to
// 78, lse is off by up to 4e-3 (8e-4 in the mean square), where it is 2e-5 below kPromptFine.
// The output keeps the error of values and probabilities in f16: 2.8e-4 to 4.0e-4 of an
// f16 output, 7e-4 in those rows; 2.1e-4 of it is the output's own rounding.
//
// Work: an item is 256 rows (two tiles of 128; row = token * heads of the key
// head + head) of one sequence and key head, over the tiles of 128 keys that they
// see.  Tiles are counted along all items, one more for an item's own cost; every
// block takes the same count of consecutive ones.  An item that blocks share
// leaves its rows' sums in the workspace, joined by kv4_prompt_join_kernel.
// (Whole items to a block, 2048 tokens on 8192 keys, 32 heads of 128, 256 items on 152
// multiprocessors: 258 us when shared ones took 254 with their join; 253 now, 0.95
// PFLOP/s where a plain product of matrices reaches 1.9.  With few items it is what
// fills the card.)
// Roles of a block's 16 warps (152 registers a thread in warps 0-7, 104 in the
// others: 2 * 152 + 2 * 104 = the 4 * 128 of the launch):
//   0-3, 4-7  softmax of tile 0, 1: a thread a row, 32 scores at a time from
//             tensor memory, P back over the scores
//   8-11      decoders: a thread a key, rows loaded a tile ahead into
//             registers, f16 core matrices (8 rows of 16 bytes) to shared memory
//   12        issues the products: PV0(i), S0(i+1), then PV1(i), S1(i+1), so that
//             one tile's softmax runs under the other tile's products; 13-15 idle
// Core matrices: K [dims/8][128 keys][8 dims] (K-major), V the same (dims along
// N: MN-major), Q like K; the order of dims within and of groups of eight is the one
// that unpacking gives, and is undone in Q's rows and the output's columns.
//
// Values out of the ordinary: a key whose steps reach 2^12 is decoded 2^-4
// smaller, and its scores or probabilities multiplied by 16 (a row that sees such a
// value keeps 2^4 more room under f16's top); a group whose step
// is not finite is decoded as zeros and marks the rows that see it, whose
// outputs of that group are NaN.
#pragma once

#include <climits>
#include <type_traits>

#include "qb_kv4.cuh"
#include "qb_tcgen05.cuh"

namespace qb {

constexpr int kPromptTile = 128;    // keys a tile, rows a tile
constexpr int kPromptQ = 2;         // row tiles an item
constexpr int kPromptRows = kPromptTile * kPromptQ;
constexpr int kPromptThreads = 16 * 32;

struct PromptK {
    Kv4AttnArgs a;
    int grp;
    int min_share;  // tiles a block
    float *part;    // [grid][2][kPromptRows][DP]: a block's pieces (0: of an item begun before it)
    float2 *stat;   // [grid][2][kPromptRows] m of the probabilities, sum
    int *last;      // [grid] the last block that holds a piece of the item that starts here and goes on; -1: none
    int4 *meta;     // [grid] that item's first token, tokens, key head, row pair
};

// A block's piece of an item: tiles t0 .. t0 + n - 1.  Every warp has its own in
// shared memory, so that walking along the block's share costs the loops no registers.
struct PromptItem {
    int s, row, len, T, q0, kvh, rp;
    int u;               // the piece's first tile, from the item's first on
    int t0, n;
    int place, rest;     // of the piece's first tile in the block's share; tiles of the item from there on
    int count;           // places of the block's share
    int from_start;
    int fine;            // keys as two f16
};

constexpr int kPromptFine = 2048;  // keys; see above
constexpr int kPromptCost = 1;  // what an item costs beside its tiles, in tiles

template <int DP>
struct PromptSmem {
    static constexpr int kTileBytes = kPromptTile * DP * 2;
    alignas(128) uint8_t q[kPromptQ][kTileBytes];
    alignas(128) uint8_t k[2][kTileBytes];
    alignas(128) uint8_t v[2][kTileBytes];
    uint16_t flags[4][kPromptTile];  // of a tile's keys: 1 K, 2 V decoded 2^-4 smaller; from bit 8 the groups that are not finite
    uint32_t any[4][4];              // whether a decoder warp's keys have one
    uint64_t q_full[kPromptQ], q_free[kPromptQ], s_full[kPromptQ], p_ready[kPromptQ], o_done[kPromptQ];
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2], drained;
    uint32_t tmem;
    long long chunk_sum[8192 / 32 + 1];
    long long x0, share;             // the block's share: its first place, its places
    PromptItem it[kPromptThreads / 32];
};

__device__ __forceinline__ float prompt_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t prompt_half2(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }

// Eight codes as f16 pairs (0,4) (1,5) (2,6) (3,7) of a word's nibbles: (code - 8) * step.
__device__ __forceinline__ uint4 prompt_decode(const CentreK &ck, uint32_t w, __half2 step) {
    const uint32_t b[4] = {centre_lo(ck, w), centre_hi(ck, w), centre_lo(ck, w >> 8), centre_hi(ck, w >> 8)};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = prompt_half2(__hmul2_rn(*reinterpret_cast<const __half2 *>(&b[i]), step));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// What that rounding left, exactly.
__device__ __forceinline__ uint4 prompt_decode_rest(const CentreK &ck, uint32_t w, __half2 step) {
    const uint32_t b[4] = {centre_lo(ck, w), centre_hi(ck, w), centre_lo(ck, w >> 8), centre_hi(ck, w >> 8)};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 c = *reinterpret_cast<const __half2 *>(&b[i]);
        o[i] = prompt_half2(__hfma2(c, step, __hneg2(__hmul2_rn(c, step))));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The whole warp's wait: false (for all of it) if any lane's ran out.
__device__ __forceinline__ bool prompt_wait(uint64_t *bar, uint32_t parity, int *fault) {
    const bool ok = mbar_try_wait(bar, parity) || mbar_wait_sleep(bar, parity, fault);
    return __all_sync(0xFFFFFFFFu, ok);
}

// The flags among the keys lo..hi of a step, together.
__device__ __forceinline__ uint32_t prompt_flags(const uint16_t *flags, int lo, int hi) {
    uint32_t all = 0;
    for (int i = max(lo, 0); i <= min(hi, kPromptTile - 1); ++i) all |= flags[i];
    return all;
}

// The probability of the maximum that m was taken from is 2^kPromptTop or, as m rises by
// whole numbers, up to twice that, and m rises when one would pass 2^kPromptMost (f16
// ends at 2^16).
constexpr float kPromptTop = 11.0f, kPromptMost = 15.9f;

// What a row's softmax carries from tile to tile.
struct PromptRow {
    float cs, m, l;   // factor of the scores, m of the probabilities, sum
    float up;         // 4 where the row sees a key of the step whose probability is 16 times larger
    int lo, hi;       // columns lo..hi of the step are seen
};

// m rises to mn in lanes where that is more, by a whole number but from -infinity: O (DP
// columns, if any products were added), the `done` columns of this step's probabilities and
// the sums l and `sum` shrink by a power of two, so that no probability is rounded again but
// below f16's normal numbers; nothing of the other lanes changes, whose rows keep their bits.
// (Its loops are not unrolled, as it is there six times: 256 -> 253 us.)
template <int DP>
__device__ __forceinline__ bool prompt_rescale(uint32_t tS, uint32_t tO, int done, float &m, float &l, uint64_t &sum,
                                                   float mn, bool have_o, uint64_t *o_done, uint32_t parity, int *fault) {
    const float al = mn == m ? 1.0f : prompt_ex2(rintf(m - mn));
    l *= al;
    sum = mul_f32x2(sum, pair_f32(al, al));
    m = mn;
    if (have_o) {
        if (!prompt_wait(o_done, parity, fault)) return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            tc_ld32(tO + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
            tc_st32(tO + 32 * c, o);
        }
    }
    if (done) {
        tc_wait_st();
        // in two factors: f16 holds none below 2^-24
        const __half2 a2 = __float2half2_rn(fmaxf(al, 0x1p-14f)), b2 = __float2half2_rn(fminf(al * 0x1p14f, 1.0f));
#pragma unroll 1
        for (int c = 0; c < done; c += 32) {  // 16 or 48 columns: the rest of the last 32 is scores, kept
            uint32_t o[32];
            tc_ld32(tS + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < done) o[i] = prompt_half2(__hmul2(__hmul2(*reinterpret_cast<const __half2 *>(&o[i]), a2), b2));
            if (done - c >= 32) {
                tc_st32(tS + c, o);
            } else {
                uint32_t h[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) h[i] = o[i];
                tc_st16(tS + c, h);
            }
        }
    }
    return true;
}

// A tile's row: 128 scores in tensor memory, 32 at a time (the next ones on
// their way), become probabilities 2^(s cs - m) as f16 over them (32 scores'
// columns have been read when the 16 columns of their probabilities are
// written).  MASKED: scores outside columns lo..hi count as -infinity; ODD:
// flagged keys' scores or probabilities are 16 times larger.
// (The loop over pairs of 32 is not unrolled: its body stays in the instruction cache.)
template <int DP, bool MASKED, bool ODD>
__device__ __forceinline__ bool prompt_step(uint32_t tS, uint32_t tO, PromptRow &row, const uint16_t *flags, bool have_o,
                                            uint64_t *o_done, uint32_t parity, int *fault) {
    uint32_t s0[32], s1[32];
    const uint64_t cs2 = pair_f32(row.cs, row.cs);
    uint64_t sum = 0;  // (0, 0)
    bool ok = true;
    auto special = [&](uint32_t (&x)[32], int c) {
        if (ODD || MASKED) {
            const int lo = row.lo - 32 * c, hi = row.hi - 32 * c;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (ODD && (flags[32 * c + i] & 1)) x[i] = __float_as_uint(__uint_as_float(x[i]) * 16.0f);
                if (i > hi || i < lo) x[i] = 0xFF800000u;
            }
        }
    };
    auto chunk = [&](uint32_t (&x)[32], uint32_t (&next)[32], int c) {
        tc_ld_wait(x);
        if (c < 3) tc_ld32_begin(tS + 32 * (c + 1), next);
        special(x, c);
        float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
        for (int i = 2; i < 32; i += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[i]));
            t1 = fmaxf(t1, __uint_as_float(x[i + 1]));
        }
        const float z = fmaxf(t0, t1) * row.cs + (ODD ? row.up : 0.0f);
        if (__any_sync(0xFFFFFFFFu, z > row.m + kPromptMost)) {
            // no score stays in a register meanwhile: they are read again
            tc_ld_wait(next);
            const float mn = !(z > row.m + kPromptMost) ? row.m
                             : row.m == -INFINITY       ? z - kPromptTop : row.m + floorf(z - kPromptTop - row.m);
            ok = prompt_rescale<DP>(tS, tO, 16 * c, row.m, row.l, sum, mn, have_o, o_done, parity, fault) && ok;
            tc_ld32_begin(tS + 32 * c, x);
            tc_ld_wait(x);
            if (c < 3) tc_ld32_begin(tS + 32 * (c + 1), next);
            special(x, c);
        }
        const float mm = row.m == -INFINITY ? 0.0f : -row.m;
        const uint64_t m2 = pair_f32(mm, mm);
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float2 y = unpair_f32(fma_f32x2(pair_f32(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), cs2, m2));
            float e0 = prompt_ex2(y.x), e1 = prompt_ex2(y.y);
            sum = add_f32x2(sum, pair_f32(e0, e1));
            if (ODD) {
                if (flags[32 * c + i] & 2) e0 *= 16.0f;
                if (flags[32 * c + i + 1] & 2) e1 *= 16.0f;
            }
            pk[i / 2] = prompt_half2(__floats2half2_rn(e0, e1));
        }
        tc_st16(tS + 16 * c, pk);
    };
    tc_ld32_begin(tS, s0);
#pragma unroll
    for (int i = 0; i < 32; ++i) s1[i] = 0u;  // begun below; named here for the compiler
#pragma unroll 1
    for (int c = 0; c < 4; c += 2) {
        chunk(s0, s1, c);
        chunk(s1, s0, c + 1);
    }
    const float2 part = unpair_f32(sum);
    row.l += part.x + part.y;
    return ok;
}

// ---- the work.  An item's place on the line of tiles: kPromptCost, then its own

__device__ __forceinline__ int prompt_pairs(const PromptK &p, int T) { return (T * p.grp + kPromptRows - 1) / kPromptRows; }

// An item's first tile and its tiles (one at least, should it see no key).
__device__ __forceinline__ int prompt_tiles(const PromptK &p, int len, int T, int rp, int &t0) {
    const int j_lo = rp * kPromptRows / p.grp, j_hi = min(T - 1, (rp * kPromptRows + kPromptRows - 1) / p.grp);
    const int pos_lo = len - T + j_lo, pos_hi = len - T + j_hi;
    t0 = kv_first_seen(pos_lo, p.a.window) / kPromptTile;
    return max(1, pos_hi < 0 ? 0 : pos_hi / kPromptTile + 1 - t0);
}

// The places of a chunk of 32 sequences, a lane's own, by the whole warp: a lane
// counts its own sequence's row pairs, or the warp one sequence after the other where
// that takes fewer steps (32 sequences of a row pair: 19 us one after the other, counted
// twice).
__device__ __forceinline__ long long prompt_places(const PromptK &p, int c, int lane, bool report, SeqInfo &q) {
    q = seq_info(p.a, c * 32 + lane, report);
    uint32_t left = __ballot_sync(0xFFFFFFFFu, q.T > 0);
    const int pairs = prompt_pairs(p, q.T), most = (int)__reduce_max_sync(0xFFFFFFFFu, (uint32_t)pairs);
    long long mine = 0;
    int t0;
    if (most <= 4 * __popc(left)) {
        for (int rp = 0; rp < pairs; ++rp) mine += prompt_tiles(p, q.len, q.T, rp, t0) + kPromptCost;
        return mine * p.a.c.nkv;
    }
    for (; left; left &= left - 1) {
        const int l = __ffs(left) - 1;
        const int len = __shfl_sync(0xFFFFFFFFu, q.len, l), T = __shfl_sync(0xFFFFFFFFu, q.T, l);
        long long n = 0;
        for (int rp = lane; rp < prompt_pairs(p, T); rp += 32) n += prompt_tiles(p, len, T, rp, t0) + kPromptCost;
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (lane == l) mine = n * p.a.c.nkv;
    }
    return mine;
}

__device__ __forceinline__ void prompt_count(const PromptK &p, int c, int lane, long long *chunk_sum) {
    SeqInfo q;
    long long n = prompt_places(p, c, lane, blockIdx.x == 0, q);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (lane == 0) chunk_sum[c] = n;
}

// By warp 0: the chunks' sums become their first places, and the block's share begins
// at a tile of an item.
__device__ __forceinline__ void prompt_find(const PromptK &p, int lane, int nchunks, long long *chunk_sum,
                                                long long &x0_out, long long &share_out, PromptItem &out) {
    long long total = 0;
    for (int c0 = 0; c0 < nchunks; c0 += 32) {
        const long long n = c0 + lane < nchunks ? chunk_sum[c0 + lane] : 0;
        long long sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        if (c0 + lane < nchunks) chunk_sum[c0 + lane] = total + sum - n;
        total += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    __syncwarp();
    long long share = (total + gridDim.x - 1) / gridDim.x;
    if (share < p.min_share) share = p.min_share;
    const long long x0 = min(blockIdx.x * share, total);
    PromptItem it = {};
    it.count = (int)(min(x0 + share, total) - x0);
    if (it.count > 0) {
        int lo = 0, hi = nchunks;  // the chunk that holds place x0
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (chunk_sum[m] <= x0) lo = m; else hi = m;
        }
        SeqInfo q;
        const long long n = prompt_places(p, lo, lane, false, q);
        long long sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        const long long before = chunk_sum[lo] + sum - n;
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, n > 0 && before <= x0);
        const int l = 31 - __clz(ok);
        long long rem = x0 - __shfl_sync(0xFFFFFFFFu, before, l);
        it.s = lo * 32 + l;
        it.row = __shfl_sync(0xFFFFFFFFu, q.row, l);
        it.len = __shfl_sync(0xFFFFFFFFu, q.len, l);
        it.T = __shfl_sync(0xFFFFFFFFu, q.T, l);
        it.q0 = __shfl_sync(0xFFFFFFFFu, q.q0, l);
        const long long per_head = __shfl_sync(0xFFFFFFFFu, n, l) / p.a.c.nkv;
        it.kvh = (int)(rem / per_head);
        rem -= it.kvh * per_head;
        for (int rp0 = 0; rp0 < prompt_pairs(p, it.T); rp0 += 32) {  // the row pair, 32 at a time
            int t0;
            const int w = rp0 + lane < prompt_pairs(p, it.T) ? prompt_tiles(p, it.len, it.T, rp0 + lane, t0) + kPromptCost : 0;
            long long end = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xFFFFFFFFu, end, o);
                if (lane >= o) end += y;
            }
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, end > rem);
            if (past) {
                const int l2 = __ffs(past) - 1;
                rem -= __shfl_sync(0xFFFFFFFFu, end - w, l2);
                it.rp = rp0 + l2;
                break;
            }
            rem -= __shfl_sync(0xFFFFFFFFu, end, 31);
        }
        // now `rem` is the place in the item
        it.u = max(0, (int)rem - kPromptCost);
        it.place = max(0, kPromptCost - (int)rem);
    }
    if (lane == 0) {
        x0_out = x0;
        share_out = share;
        out = it;
    }
}

// The block's next piece (n = 0 before the first): false when its share is done.
__device__ __forceinline__ bool prompt_next(const PromptK &p, int lane, PromptItem &io) {
    PromptItem it = io;
    __syncwarp();
    if (it.place + it.n >= it.count) return false;
    if (it.n) {  // past the piece before, which ended its item
        it.place += it.n + kPromptCost;
        if (it.place >= it.count) return false;
        it.u = 0;
        if (++it.rp == prompt_pairs(p, it.T)) {
            it.rp = 0;
            if (++it.kvh == p.a.c.nkv) {
                it.kvh = 0;
                SeqInfo q;
                do q = seq_info(p.a, ++it.s, false);
                while (q.T == 0 && it.s < p.a.s.nseq);
                it.row = q.row;
                it.len = q.len;
                it.T = q.T;
                it.q0 = q.q0;
            }
        }
    }
    int t0;
    const int tiles = prompt_tiles(p, it.len, it.T, it.rp, t0);
    it.t0 = t0 + it.u;
    it.rest = tiles - it.u;
    it.n = min(it.rest, it.count - it.place);
    it.from_start = it.u == 0;
    const int seen = it.len - it.T + it.rp * kPromptRows / p.grp + 1;  // by the first row
    it.fine = (p.a.window ? min(seen, p.a.window) : seen) < kPromptFine;
    if (lane == 0) io = it;
    __syncwarp();
    return true;
}

template <int DP>
__global__ void __launch_bounds__(kPromptThreads, 1) kv4_prompt_kernel(const PromptK p) {
    constexpr int NG = DP / 32, W = NG < 4 ? NG : 4;  // groups; one plane (DP <= 128)
    constexpr int kOctStride = kPromptTile * 16;      // bytes between groups of eight dims
    extern __shared__ uint8_t smem_raw[];
    PromptSmem<DP> &sm = *reinterpret_cast<PromptSmem<DP> *>(
        smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kPromptQ; ++i) {
            mbar_init(&sm.q_full[i], kPromptTile);
            mbar_init(&sm.q_free[i], 4);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_ready[i], kPromptTile);
            mbar_init(&sm.o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.k_free[i], 1);
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.v_free[i], 1);
        }
        mbar_init(&sm.drained, 1);
        fence_mbar_init();
    }
    if (warp == 12) {
        tc_alloc(&sm.tmem, 512);
        tc_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- the work: the block's share of the line of tiles
    const int nchunks = (p.a.s.nseq + 31) / 32;
    for (int c = warp; c < nchunks; c += kPromptThreads / 32) prompt_count(p, c, lane, sm.chunk_sum);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) prompt_find(p, lane, nchunks, sm.chunk_sum, sm.x0, sm.share, sm.it[0]);
    __syncthreads();
    if (warp > 0 && lane == 0) sm.it[warp] = sm.it[0];
    __syncthreads();  // warp 0 goes on in its own after the others have copied it
    const uint32_t tb = sm.tmem;
    PromptItem &it = sm.it[warp];
    // 128 registers a thread of 4 warpgroups at launch: 152 + 152 + 104 + 104 = 4 * 128
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        // ================================================= softmax
        const int q = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tb + lanes + 128u * q, tO = tb + lanes + 256u + (uint32_t)DP * q;
        uint32_t tiles = 0, items = 0;  // of this row tile so far
        int goes_on = -1;
        bool ok = true;
        while (ok && prompt_next(p, lane, it)) {
            const int rho = it.rp * kPromptRows + q * kPromptTile + r, j = rho / p.grp;
            const bool live = j < it.T;
            const int pos = live ? it.len - it.T + j : -1;
            const int first = kv_first_seen(pos, p.a.window);
            const int64_t tok = it.q0 + j;
            const int head = it.kvh * p.grp + rho - j * p.grp;
            const int64_t at = tok * p.a.out_stride + (int64_t)head * p.a.c.d;  // of the row's output
            float cs = 0.0f;
            {
                // The queries as f16, a row's largest magnitude scaled into [2^8, 2^9).  Four
                // lanes load a row (64 bytes together), a warp its 32 rows in four goes, all
                // loads under way together.  (A row a thread: 32 cache lines a load, 2.5 us an item.)
                constexpr int NO = DP / 32;  // eights of a row that a lane has
                uint4 raw[4][NO];
                const bool f16 = p.a.type == QB_T_F16;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int rho2 = it.rp * kPromptRows + q * kPromptTile + (r & 96) + 8 * k + (lane >> 2), j2 = rho2 / p.grp;
                    const uint16_t *src = static_cast<const uint16_t *>(p.a.q) + (it.q0 + (int64_t)j2) * p.a.q_stride +
                                          (int64_t)(it.kvh * p.grp + rho2 - j2 * p.grp) * p.a.c.d;
#pragma unroll
                    for (int o = 0; o < NO; ++o) {
                        const int el = (4 * o + (lane & 3)) * 8;
                        raw[k][o] = make_uint4(0u, 0u, 0u, 0u);
                        if (j2 < it.T && el < p.a.c.d) raw[k][o] = *reinterpret_cast<const uint4 *>(src + el);
                    }
                }
                auto load = [&](const uint4 &u, float (&x)[8]) {
                    if (f16) unpack8<QB_T_F16>(u, x); else unpack8<QB_T_BF16>(u, x);
                };
                // the item before: every warp has read its outputs from where the queries go
                if (items && !(ok = prompt_wait(&sm.q_free[q], (items - 1) & 1, p.a.fault))) break;
                ++items;
                int e = 0;  // of this thread's row
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float top = 0.0f;
#pragma unroll
                    for (int o = 0; o < NO; ++o) {
                        float x[8];
                        load(raw[k][o], x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                    const int e2 = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 8;
                    const float f = copysignf(__uint_as_float((uint32_t)(127 + 8 - e2) << 23), p.a.scale);
                    const int own = __shfl_sync(0xFFFFFFFFu, e2, 4 * (lane & 7));
                    if (lane >> 3 == k) e = own;
                    uint8_t *dst = sm.q[q] + ((r & 96) + 8 * k + (lane >> 2)) * 16;
#pragma unroll
                    for (int o = 0; o < NO; ++o) {
                        float x[8];
                        load(raw[k][o], x);
                        uint4 u;
                        u.x = prompt_half2(__floats2half2_rn(x[0] * f, x[4] * f));
                        u.y = prompt_half2(__floats2half2_rn(x[1] * f, x[5] * f));
                        u.z = prompt_half2(__floats2half2_rn(x[2] * f, x[6] * f));
                        u.w = prompt_half2(__floats2half2_rn(x[3] * f, x[7] * f));
                        *reinterpret_cast<uint4 *>(dst + (4 * o + (lane & 3)) * kOctStride) = u;
                    }
                }
                // not zero, so that a score that is masked stays -inf
                cs = fmaxf(fabsf(p.a.scale) * 1.4426950408889634f * exp2f((float)(e - 8)), 1e-37f);
                fence_async_shared();
                mbar_arrive(&sm.q_full[q]);
            }
            // tiles whose keys all of this row tile's rows see need no mask
            const int j_lo = (it.rp * kPromptRows + q * kPromptTile) / p.grp;
            const int j_hi = min(it.T - 1, (it.rp * kPromptRows + q * kPromptTile + kPromptTile - 1) / p.grp);
            const int pos_lo = j_lo < it.T ? it.len - it.T + j_lo : INT_MAX;  // no row: whatever comes out
            const int first_hi = j_lo < it.T ? kv_first_seen(it.len - it.T + j_hi, p.a.window) : 0;
            PromptRow row = {cs, -INFINITY, 0.0f, 0.0f, 0, 0};
            uint32_t bad = 0;
            const int n_tiles = it.n, t_first = it.t0;
            for (int i = 0; i < n_tiles; ++i, ++tiles) {
                const int k0 = (t_first + i) * kPromptTile;
                if (!(ok = prompt_wait(&sm.s_full[q], tiles & 1, p.a.fault))) break;
                tc_fence_after();
                const uint32_t sl = tiles & 3, par = (tiles - 1) & 1;
                const bool odd = (sm.any[sl][0] | sm.any[sl][1] | sm.any[sl][2] | sm.any[sl][3]) != 0;
                const bool masked = k0 + kPromptTile - 1 > pos_lo || k0 < first_hi;
                const uint16_t *flags = sm.flags[sl];
                row.hi = pos - k0;
                row.lo = first - k0;
                if (odd) {
                    const uint32_t fl = prompt_flags(flags, row.lo, row.hi);
                    bad |= fl >> 8;
                    row.up = fl & 2u ? 4.0f : 0.0f;
                    ok = prompt_step<DP, true, true>(tS, tO, row, flags, i > 0, &sm.o_done[q], par, p.a.fault);
                } else if (masked) {
                    ok = prompt_step<DP, true, false>(tS, tO, row, flags, i > 0, &sm.o_done[q], par, p.a.fault);
                } else {
                    ok = prompt_step<DP, false, false>(tS, tO, row, flags, i > 0, &sm.o_done[q], par, p.a.fault);
                }
                if (!ok) break;
                tc_wait_st();
                tc_fence_before();
                mbar_arrive(&sm.p_ready[q]);
            }
            const float m = row.m, l = row.l;
            if (!ok) break;
            if (!(ok = prompt_wait(&sm.o_done[q], (tiles - 1) & 1, p.a.fault))) break;
            tc_fence_after();
            const bool whole = it.from_start && it.n == it.rest;
            const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
            const int64_t rec = (int64_t)(blockIdx.x * 2 + (it.from_start ? 1 : 0)) * kPromptRows + q * kPromptTile + r;
            // The rows go through shared memory, where the queries were, so that lanes write a
            // row's bytes together: whole rows in the output's type, a piece's sums in f32 and
            // two goes of 16 dims a group.  Pieces of 16 bytes of a row lie in the order of
            // their number ^ (row % 8).  (A row a thread: 4 and 7 us an item.)
            constexpr int C = DP / 8;  // such pieces, lanes that write a row
            uint8_t *const rows = sm.q[q] + (r & 96) * DP * 2;  // this warp's 32
            const int64_t mine = live ? at : -1;
            auto piece = [&](int row2, int c) { return reinterpret_cast<uint4 *>(rows + row2 * DP * 2 + (c ^ (row2 & 7)) * 16); };
            // 32 columns are chunks 2kk, 2kk + 1 (W = 4; all four of W = 2's eight dims): eight dims of every group
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                uint32_t o[32];
                __syncwarp();
                tc_ld32(tO + 32 * kk, o);
                // column (c * (W / 2) + u) * 8 + 2 j + h is dim (2 u + h) * 32 + 4 c + j
                constexpr int CPL = 8 / W;  // chunks in 32 columns
#pragma unroll
                for (int G = 0; G < W; ++G) {
                    float x[4 * CPL];
#pragma unroll
                    for (int c = 0; c < CPL; ++c)
#pragma unroll
                        for (int j2 = 0; j2 < 4; ++j2) {
                            const float y = __uint_as_float(o[(c * (W / 2) + (G >> 1)) * 8 + 2 * j2 + (G & 1)]) * inv;
                            x[c * 4 + j2] = (bad >> G & 1) ? __uint_as_float(kEngineNaN) : y;
                        }
                    const int el = kk * 4 * CPL;  // of the group's 32
#pragma unroll
                    for (int h = 0; h < 4 * CPL; h += 8) {
                        const float (&y)[8] = *reinterpret_cast<const float (*)[8]>(&x[h]);
                        if (!whole) {
                            *reinterpret_cast<float4 *>(piece(lane, G * 4 + (el + h) % 16 / 4)) = make_float4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<float4 *>(piece(lane, G * 4 + (el + h) % 16 / 4 + 1)) = make_float4(y[4], y[5], y[6], y[7]);
                        } else if (p.a.type == QB_T_F16) {
                            store8<QB_T_F16>(piece(lane, G * 4 + (el + h) / 8), y);
                        } else {
                            store8<QB_T_BF16>(piece(lane, G * 4 + (el + h) / 8), y);
                        }
                    }
                }
                if (!whole && (kk + 1) * 4 * CPL % 16 == 0) {
                    __syncwarp();
                    float *const to = p.part + (rec - lane) * DP + (kk + 1) * 4 * CPL - 16;
#pragma unroll 4
                    for (int k = 0; k < C; ++k) {
                        const int row2 = k * (32 / C) + lane / C, c = lane % C;
                        *reinterpret_cast<uint4 *>(to + row2 * DP + c / 4 * 32 + c % 4 * 4) = *piece(row2, c);
                    }
                }
            }
            __syncwarp();
            if (whole) {
#pragma unroll 4
                for (int k = 0; k < C; ++k) {
                    const int row2 = k * (32 / C) + lane / C, c = lane % C;
                    const int64_t to = __shfl_sync(0xFFFFFFFFu, mine, row2);
                    if (to >= 0 && c * 8 < p.a.c.d)
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.a.out) + to + c * 8) = *piece(row2, c);
                }
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&sm.q_free[q]);
            if (live && !whole) p.stat[rec] = make_float2(m, l);
            if (live && whole && p.a.lse) p.a.lse[tok * p.a.nh + head] = (m + log2f(l)) * 0.6931471805599453f;
            if (threadIdx.x == 0 && it.from_start && !whole) {
                goes_on = (int)((sm.x0 + it.place + it.rest - 1) / sm.share);  // the block that holds the item's last tile
                p.meta[blockIdx.x] = make_int4(it.q0, it.T, it.kvh, it.rp);
            }
            __syncwarp();
            tc_fence_before();  // the reads of O, before the next item's products
        }
        if (threadIdx.x == 0) p.last[blockIdx.x] = ok ? goes_on : -1;
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // ================================================= decoders: a thread a key
        const CentreK ck;
        const int r = threadIdx.x - 8 * 32, dw = warp - 8;
        const int page = p.a.c.page, code_bytes = page * DP / 2, step_bytes = page * DP / 16;
        uint32_t kt = 0, fill = 0;  // key tiles, fills of K's buffers so far
        bool ok = true;
        constexpr int NV = DP / 32;  // 16-byte pieces of a row's codes
        uint4 kx[NV], vx[NV];
        uint32_t ks[NG / 2], vs[NG / 2];
        while (ok && prompt_next(p, lane, it)) {
            auto load = [&](int tile, uint4 (&kc)[NV], uint32_t (&kst)[NG / 2], uint4 (&vc)[NV], uint32_t (&vst)[NG / 2]) {
                const int key = tile * kPromptTile + r;
                if (key < it.len) {
                    int pg = p.a.s.tables[(int64_t)it.row * p.a.s.maxp + (key >> p.a.c.pshift)];
                    if ((uint32_t)pg >= (uint32_t)p.a.c.npages) {
                        atomicOr(p.a.fault, kFaultIndex);
                        pg = 0;
                    }
                    const int rr = key & (page - 1);
                    const uint8_t *b = p.a.c.data + ((int64_t)pg * p.a.c.nkv + it.kvh) * p.a.c.block_bytes;
                    const uint4 *kp = reinterpret_cast<const uint4 *>(b + rr * 16 * W);
                    const uint4 *vp = reinterpret_cast<const uint4 *>(b + code_bytes + step_bytes + rr * 16 * W);
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        kc[i] = kp[i];
                        vc[i] = vp[i];
                    }
                    const uint32_t *kst_p = reinterpret_cast<const uint32_t *>(b + code_bytes + rr * NG * 2);
                    const uint32_t *vst_p = reinterpret_cast<const uint32_t *>(b + 2 * code_bytes + step_bytes + rr * NG * 2);
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i) {
                        kst[i] = kst_p[i];
                        vst[i] = vst_p[i];
                    }
                } else {  // no key: zeros
#pragma unroll
                    for (int i = 0; i < NV; ++i) kc[i] = vc[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
#pragma unroll
                    for (int i = 0; i < NG / 2; ++i) kst[i] = vst[i] = 0u;
                }
            };
            load(it.t0, kx, ks, vx, vs);
            const bool fine = it.fine != 0;
            for (int i = 0; i < it.n; ++i, ++kt) {
                const int slot = kt & 1;
                const uint32_t ph = (kt >> 1) & 1;
                uint4 kc[NV], vc[NV];
                uint32_t kst[NG / 2], vst[NG / 2];
#pragma unroll
                for (int i2 = 0; i2 < NV; ++i2) {
                    kc[i2] = kx[i2];
                    vc[i2] = vx[i2];
                }
#pragma unroll
                for (int i2 = 0; i2 < NG / 2; ++i2) {
                    kst[i2] = ks[i2];
                    vst[i2] = vs[i2];
                }
                if (i + 1 < it.n) load(it.t0 + i + 1, kx, ks, vx, vs);
                // what is out of the ordinary
                const int rr = ((it.t0 + i) * kPromptTile + r) & (page - 1);
                uint32_t fl = 0;
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    const uint32_t kb = (kst[G / 2] >> (16 * (G & 1))) & 0x7FFFu, vb = (vst[G / 2] >> (16 * (G & 1))) & 0x7FFFu;
                    if (kb >= 0x6C00u) fl |= 1u;  // 2^12
                    if (vb >= 0x7C00u) fl |= 256u << G;
                    else if (vb >= 0x6C00u) fl |= 2u;
                }
                const __half2 sixteenth = __float2half2_rn(0.0625f);
                if (fl) {
#pragma unroll
                    for (int h = 0; h < NG / 2; ++h) {
                        __half2 &a = *reinterpret_cast<__half2 *>(&kst[h]), &b = *reinterpret_cast<__half2 *>(&vst[h]);
                        if (fl & 1u) a = __hmul2(a, sixteenth);
                        if (fl >> 8 >> (2 * h) & 1u) vst[h] &= 0xFFFF0000u;
                        if (fl >> 8 >> (2 * h + 1) & 1u) vst[h] &= 0x0000FFFFu;
                        if (fl & 2u) b = __hmul2(b, sixteenth);
                    }
                }
                if (!(ok = prompt_wait(&sm.k_free[fill & 1], (fill >> 1 & 1) ^ 1u, p.a.fault))) break;
                // the tile's flags: three tiles at most are in use, four are held
                sm.flags[kt & 3][r] = (uint16_t)fl;
                const uint32_t any = __ballot_sync(0xFFFFFFFFu, fl != 0);
                if (lane == 0) sm.any[kt & 3][dw] = any;
                uint8_t *dst = sm.k[fill & 1] + r * 16;
                auto keys = [&](auto rest) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int gi = 0; gi < W; ++gi) {
                            const int wi = t * W + gi;  // the row's word: elements 8 t .. of group gi
                            const uint4 &u = kc[wi / 4];
                            const uint32_t w = wi % 4 == 0 ? u.x : wi % 4 == 1 ? u.y : wi % 4 == 2 ? u.z : u.w;
                            const __half2 sp = *reinterpret_cast<const __half2 *>(&kst[gi / 2]);
                            const __half2 step = (gi & 1) ? __high2half2(sp) : __low2half2(sp);
                            *reinterpret_cast<uint4 *>(dst + (gi * 4 + t) * kOctStride) =
                                decltype(rest)::value ? prompt_decode_rest(ck, w, step) : prompt_decode(ck, w, step);
                        }
                    fence_async_shared();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.k_full[fill & 1]);
                    ++fill;
                };
                keys(std::false_type());
                if (fine) {
                    if (!(ok = prompt_wait(&sm.k_free[fill & 1], (fill >> 1 & 1) ^ 1u, p.a.fault))) break;
                    dst = sm.k[fill & 1] + r * 16;
                    if (fl & 1u) {  // an infinite step leaves nothing
#pragma unroll
                        for (int h = 0; h < NG / 2; ++h) {
                            if ((kst[h] & 0x7C00u) == 0x7C00u) kst[h] &= 0xFFFF0000u;
                            if ((kst[h] & 0x7C000000u) == 0x7C000000u) kst[h] &= 0x0000FFFFu;
                        }
                    }
                    // decoded anew: what is common to both passes would not fit the registers
#pragma unroll
                    for (int t = 0; t < NV; ++t)
                        asm volatile("" : "+r"(kc[t].x), "+r"(kc[t].y), "+r"(kc[t].z), "+r"(kc[t].w));
                    keys(std::true_type());
                }
                if (!(ok = prompt_wait(&sm.v_free[slot], ph ^ 1u, p.a.fault))) break;
                dst = sm.v[slot] + r * 16;
                const int swz = 4 * ((rr >> 1) & 1);
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int u2 = 0; u2 < W / 2; ++u2) {
                        const int wi = c * (W / 2) + u2;  // the row's word: chunk c ^ swz, groups 2 u2 and 2 u2 + 1
                        const uint4 &u = vc[wi / 4];
                        const uint32_t w = wi % 4 == 0 ? u.x : wi % 4 == 1 ? u.y : wi % 4 == 2 ? u.z : u.w;
                        *reinterpret_cast<uint4 *>(dst + ((c ^ swz) * (W / 2) + u2) * kOctStride) =
                            prompt_decode(ck, w, *reinterpret_cast<const __half2 *>(&vst[u2]));
                    }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.v_full[slot]);
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // ================================================= products
        const uint32_t idS = tc_idesc_f16(kPromptTile, false), idO = tc_idesc_f16(DP, true);
        uint32_t kt = 0, fill = 0, items = 0;  // key tiles, fills of K's buffers, items so far
        bool ok = warp == 12;
        // S = Q K^T with the key tile of fill f (and f + 1, what its rounding left)
        auto scores = [&](int q, uint32_t f, auto fine_t) {
            constexpr bool fine = decltype(fine_t)::value;
            const uint32_t qa = smem_u32(sm.q[q]);
            if (elect_one()) {
                const uint32_t ka = smem_u32(sm.k[f & 1]);
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    tc_mma_ss(tb + 128u * q, tc_desc(qa + 2 * s * kOctStride, kOctStride, 128),
                              tc_desc(ka + 2 * s * kOctStride, kOctStride, 128), idS, s != 0);
                if (fine) {
                    const uint32_t kb = smem_u32(sm.k[(f + 1) & 1]);
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s)
                        tc_mma_ss(tb + 128u * q, tc_desc(qa + 2 * s * kOctStride, kOctStride, 128),
                                  tc_desc(kb + 2 * s * kOctStride, kOctStride, 128), idS, true);
                }
                tc_commit(&sm.s_full[q]);
                if (q == kPromptQ - 1) {
                    tc_commit(&sm.k_free[f & 1]);
                    if (fine) tc_commit(&sm.k_free[(f + 1) & 1]);
                }
            }
            __syncwarp();
        };
        auto keys_there = [&](uint32_t f, auto fine_t) {
            return prompt_wait(&sm.k_full[f & 1], f >> 1 & 1, p.a.fault) &&
                   (!decltype(fine_t)::value || prompt_wait(&sm.k_full[(f + 1) & 1], (f + 1) >> 1 & 1, p.a.fault));
        };
        // O (+)= P V
        auto outputs = [&](int q, uint32_t t, bool first) {
            const uint32_t va = smem_u32(sm.v[t & 1]);
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < kPromptTile / 16; ++s)
                    tc_mma_ts(tb + 256u + (uint32_t)DP * q, tb + 128u * q + 8u * s, tc_desc(va + 256 * s, 128, kOctStride),
                              idO, !first || s != 0);
                tc_commit(&sm.o_done[q]);
                if (q == kPromptQ - 1) tc_commit(&sm.v_free[t & 1]);
            }
            __syncwarp();
        };
        auto item = [&](auto fine) {
            constexpr uint32_t step = decltype(fine)::value ? 2 : 1;
            if (!(ok = keys_there(fill, fine))) return;
            tc_fence_after();
            for (int q = 0; q < kPromptQ; ++q) scores(q, fill, fine);
            for (int i = 0; i < it.n; ++i, ++kt, fill += step) {
                const bool more = i + 1 < it.n;
                if (!(ok = prompt_wait(&sm.v_full[kt & 1], (kt >> 1) & 1, p.a.fault))) return;
                if (more && !(ok = keys_there(fill + step, fine))) return;
                for (int q = 0; q < kPromptQ; ++q) {
                    if (!(ok = prompt_wait(&sm.p_ready[q], kt & 1, p.a.fault))) return;
                    tc_fence_after();
                    outputs(q, kt, i == 0);
                    if (!more) continue;
                    // products with different accumulators are not ordered: the next scores,
                    // which go where P is, wait until it has been read
                    if (!(ok = prompt_wait(&sm.o_done[q], kt & 1, p.a.fault))) return;
                    tc_fence_after();
                    scores(q, fill + step, fine);
                }
            }
        };
        while (ok && prompt_next(p, lane, it)) {
            for (int q = 0; q < kPromptQ && ok; ++q) ok = prompt_wait(&sm.q_full[q], items & 1, p.a.fault);
            ++items;
            if (!ok) break;
            if (it.fine) item(std::true_type());
            else item(std::false_type());
        }
        // tensor and shared memory are given back after the last product, also where a wait was given up
        if (warp == 12) {
            if (elect_one()) tc_commit(&sm.drained);
            __syncwarp();
            prompt_wait(&sm.drained, 0, p.a.fault);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tc_dealloc(tb, 512);
}

constexpr int kJoinRows = 16;  // rows a block of the join

// Joins an item's pieces: block (b, y) has the item that starts at block b of the
// prompt kernel and goes on, its rows 16 y .. 16 y + 15, two to a warp, their loads
// under way together; weights 2^(m_i - m), sums in the order of the keys.
template <int DP>
__global__ void __launch_bounds__(256, 6) kv4_prompt_join_kernel(const PromptK p) {
    constexpr int E = DP / 32, RW = kJoinRows / 8;
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x;
    const int last = p.last[b];
    if (last < 0) return;
    const int4 it = p.meta[b];
    const int parts = last - b + 1, row0 = blockIdx.y * kJoinRows + warp * RW;
    if ((it.w * kPromptRows + row0) / p.grp >= it.y) return;
    auto rec = [&](int k, int r) { return (int64_t)((b + k) * 2 + (k == 0 ? 1 : 0)) * kPromptRows + row0 + r; };
    float m[RW], l[RW], acc[RW][E];
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = 0.0f;
    }
    for (int k = lane; k < parts; k += 32)
#pragma unroll
        for (int r = 0; r < RW; ++r) m[r] = fmaxf(m[r], p.stat[rec(k, r)].x);
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int o = 16; o; o >>= 1) m[r] = fmaxf(m[r], __shfl_xor_sync(0xFFFFFFFFu, m[r], o));
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
        float2 st[RW], x[RW][E / 2];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            st[r] = p.stat[rec(k, r)];
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
                x[r][e] = reinterpret_cast<const float2 *>(p.part + rec(k, r) * DP + lane * E)[e];
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const float w = prompt_ex2(st[r].x - (m[r] == -INFINITY ? 0.0f : m[r]));
            l[r] += w * st[r].y;
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                acc[r][2 * e] += w * x[r][e].x;
                acc[r][2 * e + 1] += w * x[r][e].y;
            }
        }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
        const int rho = it.w * kPromptRows + row0 + r, j = rho / p.grp;
        if (j >= it.y) continue;
        const int64_t tok = it.x + j;
        const int head = it.z * p.grp + rho - j * p.grp;
        const float inv = l[r] == 0.0f ? 0.0f : 1.0f / l[r];
        uint16_t *out = static_cast<uint16_t *>(p.a.out) + tok * p.a.out_stride + (int64_t)head * p.a.c.d + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            if (lane * E + e >= p.a.c.d) continue;
            const float y0 = acc[r][e] * inv, y1 = acc[r][e + 1] * inv;
            if (p.a.type == QB_T_F16)
                *reinterpret_cast<__half2 *>(out + e) = __floats2half2_rn(y0, y1);
            else
                *reinterpret_cast<__nv_bfloat162 *>(out + e) = __floats2bfloat162_rn(y0, y1);
        }
        if (lane == 0 && p.a.lse) p.a.lse[tok * p.a.nh + head] = (m[r] + log2f(l[r])) * 0.6931471805599453f;
    }
}

// Byte offsets of the workspace's parts.
struct PromptWs {
    int64_t part, stat, meta, last, end;
};
inline PromptWs prompt_ws(int64_t grid, int64_t dp) {
    PromptWs w;
    w.part = 0;
    w.stat = w.part + grid * 2 * kPromptRows * dp * 4;
    w.meta = w.stat + grid * 2 * kPromptRows * 8;
    w.last = w.meta + grid * 16;
    w.end = (w.last + grid * 4 + 15) / 16 * 16;
    return w;
}

template <int DP>
int launch_kv4_prompt(const Kv4AttnArgs &a, cudaStream_t stream) {
    PromptK p;
    p.a = a;
    p.grp = a.nh / a.c.nkv;
    p.min_share = 4;
    const int grid = attn_grid();
    const PromptWs w = prompt_ws(grid, DP);
    p.part = reinterpret_cast<float *>(a.ws + w.part);
    p.stat = reinterpret_cast<float2 *>(a.ws + w.stat);
    p.meta = reinterpret_cast<int4 *>(a.ws + w.meta);
    p.last = reinterpret_cast<int *>(a.ws + w.last);
    constexpr int smem = (int)sizeof(PromptSmem<DP>) + 128;
    auto *f = kv4_prompt_kernel<DP>;
    if (ensure_smem_limit(reinterpret_cast<const void *>(f), smem) != QB_OK) return QB_E_CUDA;
    if (const int rc = launch_pdl(f, dim3((unsigned)grid), dim3(kPromptThreads), smem, stream, p)) return rc;
    return launch_pdl(kv4_prompt_join_kernel<DP>, dim3((unsigned)grid, kPromptRows / kJoinRows), dim3(256), 0, stream, p);
}

}  // namespace qb
