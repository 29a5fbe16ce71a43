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
// Operands.  Codes become f16 without a conversion.  Keys: a code in the low bits
// of an f16 is the subnormal c * 2^-24, exact, so a mask is the whole unpacking;
// the -8 is the accumulator's initial value, -8 * sum of the queries.
// Values: (1024 + c) - 1032 by one packed addition (the sum of probabilities
// times 8 taken off at the end would cancel where the values' mean is small).
// Queries are scaled by a power of two a row to f16's top; in f32 they enter as
// two f16 (high and low part, 22 bits), in rows r and r + 8 of the same
// m16n8k16 product.  The probabilities times steps likewise, scaled by a power of
// two that follows the largest step seen (as the running maximum does).
//
// Layout.  A lane of the B fragment (column g, slots of t) needs 8 elements of
// key g in one word: the cache's key rows are ordered so that one wide load holds
// a lane's words of all groups; value rows so that it holds a lane's halves.
// Columns are keys in the order 0 7 1 6 2 5 3 4 (column 2t: key t, 2t + 1: key
// 7 - t), which keeps both loads free of bank conflicts.
//
// Work.  Units of 32 keys of one (sequence, key head, row tile), counted along
// the whole batch; every warp takes the same number of consecutive units
// whatever the sequences' lengths are, and streams them through its own ring of
// bulk copies (a page's block of a head is contiguous), so warps never wait for
// one another.  A piece of an item that its warp does not hold whole leaves its
// sums in the workspace, joined by kv4_combine_kernel in the order of the keys.
#pragma once

#include <climits>

#include "qb_kv4.cuh"

namespace qb {

constexpr int kStepWarps = 8;
constexpr int kUnit = 32;       // keys a unit
constexpr int kMaxRows = 16;    // rows (token, query head) of a row tile
constexpr int kSeqChunk = 32;   // sequences summed together in a block's table

template <int DP>
constexpr int step_stages() { return DP == 64 ? 8 : DP == 128 ? 6 : 3; }
template <int DP>
constexpr int step_unit_bytes() { return kv4_block(kUnit, DP); }

struct StepK {
    Kv4AttnArgs a;
    int grp;          // query heads a key head
    int nosplit;      // a worker's share is whole items
    int nworkers;
    int min_share;    // units
    float *part;      // [nworkers][2][kMaxRows][DP]
    float2 *stat;     // [nworkers][2][kMaxRows] running maximum, sum
    int4 *meta;       // [nworkers][2] of the item that starts at a worker and goes on: the last worker that
                      // holds a piece of it (-1: no such item), first token, tokens, key head; row tile
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// rows 8..15 of A and of the sums are not used
__device__ __forceinline__ void mma_f16(float (&c)[2], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
    asm volatile(
        "{\n\t.reg .f32 x, y;\n\t"
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, x, y}, {%2, %3, %4, %3}, {%5, %6}, "
        "{%0, %1, %7, %7};\n\t}"
        : "+f"(c[0]), "+f"(c[1])
        : "r"(a0), "r"(0), "r"(a2), "r"(b0), "r"(b1), "f"(0.0f));
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

// units of one item of the sequence: from the unit of its first seen key to its end (one at least)
__device__ __forceinline__ void seq_units(const SeqInfo &q, int window, int &u0, int &nu) {
    const int first = window ? max(0, q.len - q.T - window + 1) : 0;
    u0 = first / kUnit;
    nu = max(1, (q.len + kUnit - 1) / kUnit - u0);
}

// MODE 0: f32 rows (R = 8, two f16 a factor); 1: half precision, up to 8 rows; 2: half precision, 16 rows.
template <int MODE>
constexpr int step_rows() { return MODE == 2 ? 16 : 8; }

// position in the call's work
struct StepPos {
    int s, kvh, rt, u;       // sequence, key head, row tile, unit of the item
    int row, len, T, q0;     // the sequence
    int u0, nu, nrt;
    int base;                // the sequences base .. base + 31 are in the lanes' registers
    SeqInfo mine;            // lane l: sequence base + l
};

template <int R>
__device__ __forceinline__ void step_load_seq(const StepK &p, StepPos &x, int lane) {
    for (;;) {  // past sequences without new tokens
        if (x.s >= x.base + 32) {
            x.base = x.s;
            x.mine = seq_info(p.a, x.base + lane, false);
        }
        const int l = x.s - x.base;
        x.row = __shfl_sync(0xFFFFFFFFu, x.mine.row, l);
        x.len = __shfl_sync(0xFFFFFFFFu, x.mine.len, l);
        x.T = __shfl_sync(0xFFFFFFFFu, x.mine.T, l);
        x.q0 = __shfl_sync(0xFFFFFFFFu, x.mine.q0, l);
        if (x.T > 0 || x.s >= p.a.s.nseq) break;
        ++x.s;
    }
    const SeqInfo q = {x.row, x.len, x.T, x.q0};
    seq_units(q, p.a.window, x.u0, x.nu);
    x.nrt = (x.T * p.grp + R - 1) / R;
}

// the next unit; whether it begins another item
template <int R>
__device__ __forceinline__ bool step_next(const StepK &p, StepPos &x, int lane) {
    if (++x.u < x.nu) return false;
    x.u = 0;
    if (++x.rt == x.nrt) {
        x.rt = 0;
        if (++x.kvh == p.a.c.nkv) {
            x.kvh = 0;
            ++x.s;
            step_load_seq<R>(p, x, lane);
        }
    }
    return true;
}

template <int DP, int MODE, int SB>
__global__ void __launch_bounds__(kStepWarps * 32, 1) kv4_step_kernel(const StepK p) {
    constexpr int R = step_rows<MODE>(), NR = MODE == 2 ? 2 : 1;   // rows of a tile, rows of a lane
    constexpr int NC = MODE == 1 ? 2 : 4;                          // sums a lane holds of a product
    constexpr int NG = DP / 32, W = NG < 4 ? NG : 4, NP = NG / W;  // groups, groups a plane, planes
    constexpr int kStages = step_stages<DP>(), kBytes = step_unit_bytes<DP>();
    constexpr int kSub = kv4_block(SB, DP);                        // a sub-block of SB rows in shared memory
    constexpr int kCodes = SB * DP / 2, kSteps = SB * DP / 16, kPlane = SB * 16 * W;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bars[kStepWarps][kStages];
    __shared__ long long chunk_sum[8192 / kSeqChunk + 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * kStages * kBytes;
    uint64_t *full = full_bars[warp];
    if (lane < kStages) mbar_init(full + lane, 1);
    fence_mbar_init();
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();

    // ---- the work: units before each chunk of sequences
    const int nseq = p.a.s.nseq, nchunks = (nseq + kSeqChunk - 1) / kSeqChunk;
    SeqInfo mine = {0, 0, 0, 0};
    for (int c = warp; c < nchunks; c += kStepWarps) {
        const SeqInfo q = seq_info(p.a, c * kSeqChunk + lane, blockIdx.x == 0);
        if (nchunks == 1) mine = q;
        int u0, nu;
        seq_units(q, p.a.window, u0, nu);
        long long n = (long long)p.a.c.nkv * ((q.T * p.grp + R - 1) / R) * (p.nosplit ? 1 : nu);
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (lane == 0) chunk_sum[c] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        long long sum = 0;
        for (int c = 0; c < nchunks; ++c) {
            const long long n = chunk_sum[c];
            chunk_sum[c] = sum;
            sum += n;
        }
        chunk_sum[nchunks] = sum;
    }
    __syncthreads();
    const long long total = chunk_sum[nchunks];
    // workers in the order of the units: neighbours are on different multiprocessors
    const int worker = warp * gridDim.x + blockIdx.x;
    long long share = (total + p.nworkers - 1) / p.nworkers;
    if (!p.nosplit && share < p.min_share) share = p.min_share;
    const long long begin = worker * share, end = min(begin + share, total);
    if (lane == 0 && !p.nosplit) p.meta[worker * 2].x = -1;
    if (begin >= end) return;

    StepPos cur;
    cur.s = 0;
    {
        int lo = 0, hi = nchunks;  // the chunk that holds unit `begin`
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (chunk_sum[m] <= begin) lo = m; else hi = m;
        }
        cur.base = lo * kSeqChunk;
        if (nchunks == 1 && warp == 0) cur.mine = mine;
        else cur.mine = seq_info(p.a, cur.base + lane, false);
        int u0, nu;
        seq_units(cur.mine, p.a.window, u0, nu);
        const int items = p.a.c.nkv * ((cur.mine.T * p.grp + R - 1) / R);
        const long long n = (long long)items * (p.nosplit ? 1 : nu);
        long long sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        const long long before = chunk_sum[lo] + sum - n;
        // the last lane with units that starts at or before `begin`
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, n > 0 && before <= begin);
        const int l = 31 - __clz(ok);
        const long long rem = begin - __shfl_sync(0xFFFFFFFFu, before, l);
        cur.s = cur.base + l;
        step_load_seq<R>(p, cur, lane);
        const long long it = p.nosplit ? rem : rem / cur.nu;
        cur.u = p.nosplit ? 0 : (int)(rem - it * cur.nu);
        cur.kvh = (int)(it / cur.nrt);
        cur.rt = (int)(it - (long long)cur.kvh * cur.nrt);
    }

    // ---- the copies, kStages units ahead.  A lane has one piece of a unit:
    // a page (16 or 32 tokens a page), or a part of half a page (64)
    int sub = 0, src_off = 0, half_mul = 0, dst_off = 0, nbytes = 0;
    if (p.a.c.page == 64) {
        constexpr int kC64 = 64 * DP / 2, kS64 = 64 * DP / 16, kP64 = 64 * 16 * W;
        const int piece = lane % (NP + 1), side = lane / (NP + 1);
        if (lane < 2 * (NP + 1)) {
            const bool steps = piece == NP;
            nbytes = steps ? kSteps : kPlane;
            src_off = side * (kC64 + kS64) + (steps ? kC64 : piece * kP64);
            half_mul = steps ? kS64 / 2 : kP64 / 2;
            dst_off = side * (kCodes + kSteps) + (steps ? kCodes : piece * kPlane);
        }
    } else if (lane < kUnit / SB) {
        sub = lane;
        nbytes = kSub;
        dst_off = lane * kSub;
    }
    StepPos ahead = cur;
    long long left_ahead = end - begin;
    int pg = 0;  // this lane's page of the unit at `ahead`
    bool pg_there = false;
    auto find_page = [&]() {
        pg_there = false;
        if (left_ahead > 0 && nbytes) {
            const int u = ahead.u0 + ahead.u;
            const int pi = p.a.c.page == 64 ? u >> 1 : p.a.c.page == 32 ? u : 2 * u + sub;
            if ((p.a.c.page == 64 ? u * kUnit : pi * p.a.c.page) < ahead.len) {
                pg_there = true;
                pg = p.a.s.tables[(int64_t)ahead.row * p.a.s.maxp + pi];
            }
        }
    };
    int islot = 0;
    auto issue = [&]() {
        if (left_ahead > 0) {
            if (pg_there && (pg < 0 || pg >= p.a.c.npages)) {
                atomicOr(p.a.fault, kFaultIndex);
                pg = 0;
            }
            int bytes = pg_there ? nbytes : 0;
#pragma unroll
            for (int o = 4; o; o >>= 1) bytes += __shfl_xor_sync(0xFFFFFFFFu, bytes, o);  // pieces are in lanes 0..7
            if (lane == 0) mbar_arrive_expect_tx(full + islot, (uint32_t)bytes);
            __syncwarp();
            if (pg_there)
                bulk_g2s(ring + islot * kBytes + dst_off,
                         p.a.c.data + ((int64_t)pg * p.a.c.nkv + ahead.kvh) * p.a.c.block_bytes + src_off +
                             (((ahead.u0 + ahead.u) & 1) ? half_mul : 0),
                         (uint32_t)nbytes, full + islot);
            const bool item_end = step_next<R>(p, ahead, lane);
            left_ahead -= p.nosplit ? (item_end ? 1 : 0) : 1;
            find_page();
        }
        islot = islot + 1 == kStages ? 0 : islot + 1;
    };
    find_page();
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) issue();

    // ---- this lane's places in a unit
    const int key0 = t, key1 = 7 - t;                      // its columns 2t, 2t + 1 of eight keys
    const int kcol = (g & 1) ? 7 - (g >> 1) : (g >> 1);    // the key of column g
    const int koff = kcol * 16 * W + t * 4 * W;
    const int voff0 = kCodes + kSteps + key0 * 16 * W + ((g ^ (4 * (t >> 1))) * 2 * W);
    const int voff1 = kCodes + kSteps + key1 * 16 * W + ((g ^ (4 * (1 - (t >> 1)))) * 2 * W);

    long long left = end - begin;
    int slot = 0;
    uint32_t phase = 0;
    while (left > 0) {
        // ---- an item, or this worker's piece of it
        const int s_kvh = cur.kvh, s_rt = cur.rt, s_q0 = cur.q0, s_T = cur.T, s_len = cur.len, s_nu = cur.nu;
        const bool from_start = cur.u == 0;
        const long long item_left = s_nu - cur.u;  // units of the item from here on
        const int units = (int)(p.nosplit ? item_left : min(item_left, left));
        const bool to_end = units == item_left;

        // the lane's rows: token and head, place, queries as fragments
        int pos[NR], first[NR];
        int64_t otok[NR];
        int ohead[NR];
        bool live[NR];
        uint32_t A[NG][2][NR == 2 || MODE == 0 ? 4 : 2];
        float cinit[NG][MODE == 1 ? 1 : 2], cs[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int rho = s_rt * R + g + 8 * r;
            const int j = rho / p.grp;
            live[r] = j < s_T;
            pos[r] = live[r] ? s_len - s_T + j : -1;
            first[r] = p.a.window ? max(0, pos[r] - p.a.window + 1) : 0;
            otok[r] = s_q0 + j;
            ohead[r] = s_kvh * p.grp + rho - j * p.grp;
            float x[NG][8];
            float top = 0.0f;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[G][i] = 0.0f;
                if (live[r] && G * 32 + t * 8 < p.a.c.d) {
                    const int64_t at = otok[r] * p.a.q_stride + (int64_t)ohead[r] * p.a.c.d + G * 32 + t * 8;
                    if constexpr (MODE == 0) {
                        load8<QB_T_F32>(static_cast<const float *>(p.a.q) + at, x[G]);
                    } else {
                        const uint16_t *q = static_cast<const uint16_t *>(p.a.q) + at;
                        if (p.a.type == QB_T_F16) load8<QB_T_F16>(q, x[G]); else load8<QB_T_BF16>(q, x[G]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[G][i]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            // the row's largest magnitude into [2^14, 2^15)
            const int e = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 14;
            const float f = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            cs[r] = p.a.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + 10) << 23) * exp2f((float)e);
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                float hi[8], lo[8], sh = 0.0f, sl = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = x[G][i] * f;
                    hi[i] = __half2float(__float2half_rn(y));
                    lo[i] = y - hi[i];
                    sh += hi[i];
                    if (MODE == 0) {
                        lo[i] = __half2float(__float2half_rn(lo[i]));
                        sl += lo[i];
                    }
                }
                sh += __shfl_xor_sync(0xFFFFFFFFu, sh, 1);
                sh += __shfl_xor_sync(0xFFFFFFFFu, sh, 2);
                const float c8 = -8.0f / 16777216.0f;
                if constexpr (MODE == 0) {
                    sl += __shfl_xor_sync(0xFFFFFFFFu, sl, 1);
                    sl += __shfl_xor_sync(0xFFFFFFFFu, sl, 2);
                    cinit[G][0] = c8 * sh;
                    cinit[G][1] = c8 * sl;
                } else {
                    cinit[G][r] = c8 * sh;
                }
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    // codes 2m, 2m + 4 stand as c * 2^-24, codes 2m + 1, 2m + 5 as 16 c * 2^-24
                    const uint32_t a_lo = pack_f16(hi[2 * m], hi[2 * m + 4]);
                    const uint32_t a_hi = pack_f16(hi[2 * m + 1] * 0.0625f, hi[2 * m + 5] * 0.0625f);
                    if constexpr (MODE == 0) {
                        A[G][m][0] = a_lo;
                        A[G][m][2] = a_hi;
                        A[G][m][1] = pack_f16(lo[2 * m], lo[2 * m + 4]);
                        A[G][m][3] = pack_f16(lo[2 * m + 1] * 0.0625f, lo[2 * m + 5] * 0.0625f);
                    } else if constexpr (MODE == 1) {
                        A[G][m][0] = a_lo;
                        A[G][m][1] = a_hi;
                    } else {
                        A[G][m][r] = a_lo;
                        A[G][m][2 + r] = a_hi;
                    }
                }
            }
        }
        // units whose keys every row sees need no mask
        const int pos_lo = s_len - s_T + (s_rt * R) / p.grp;
        const int pos_hi = s_len - s_T + min(s_T - 1, (s_rt * R + R - 1) / p.grp);
        const int first_hi = p.a.window ? max(0, pos_hi - p.a.window + 1) : 0;

        float O[NG][4][NC];
        float m[NR], l[NR];
        int eb = 1;  // biased exponent (binary16's) of the largest step so far
#pragma unroll
        for (int G = 0; G < NG; ++G)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < NC; ++c) O[G][j][c] = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
        }

        for (int un = 0; un < units; ++un) {
            const int k0 = (cur.u0 + cur.u) * kUnit;
            const bool landed = mbar_wait_bounded(full + slot, phase, p.a.fault);
            if (!__all_sync(0xFFFFFFFFu, landed)) return;  // a copy never completed: fault word raised
            const uint8_t *ub = ring + slot * kBytes;
            const bool masked = k0 + kUnit - 1 > pos_lo || k0 < first_hi;

            // ---- scores of this lane's eight keys
            float z[4][2 * NR];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const uint8_t *kb = ub + (nt * 8 / SB) * kSub + 0;
                const int r0 = (nt * 8) % SB;
#pragma unroll
                for (int i = 0; i < 2 * NR; ++i) z[nt][i] = 0.0f;
                uint32_t st0[NG / 2], st1[NG / 2];
                lds<NG / 2>(kb + kCodes + (r0 + key0) * NG * 2, st0);
                lds<NG / 2>(kb + kCodes + (r0 + key1) * NG * 2, st1);
#pragma unroll
                for (int pl = 0; pl < NP; ++pl) {
                    uint32_t w[W];
                    lds<W>(kb + pl * kPlane + r0 * 16 * W + koff, w);
#pragma unroll
                    for (int gi = 0; gi < W; ++gi) {
                        const int G = pl * W + gi;
                        const uint32_t v = w[gi] >> 8;
                        float acc[NC];
                        if constexpr (MODE == 1) {
                            acc[0] = acc[1] = cinit[G][0];
                            mma_f16(acc, A[G][0][0], A[G][0][1], w[gi] & 0x000F000Fu, w[gi] & 0x00F000F0u);
                            mma_f16(acc, A[G][1][0], A[G][1][1], v & 0x000F000Fu, v & 0x00F000F0u);
                        } else {
                            acc[0] = acc[1] = cinit[G][0];
                            acc[2] = acc[3] = cinit[G][1];
                            mma_f16(acc, A[G][0][0], A[G][0][1], A[G][0][2], A[G][0][3], w[gi] & 0x000F000Fu,
                                    w[gi] & 0x00F000F0u);
                            mma_f16(acc, A[G][1][0], A[G][1][1], A[G][1][2], A[G][1][3], v & 0x000F000Fu,
                                    v & 0x00F000F0u);
                        }
                        const float2 d0 = unpack_f16(st0[G / 2]), d1 = unpack_f16(st1[G / 2]);
                        const float s0 = (G & 1) ? d0.y : d0.x, s1 = (G & 1) ? d1.y : d1.x;
                        z[nt][0] = fmaf(s0, acc[0], z[nt][0]);
                        z[nt][1] = fmaf(s1, acc[1], z[nt][1]);
                        if constexpr (MODE == 0) {
                            z[nt][0] = fmaf(s0, acc[2], z[nt][0]);
                            z[nt][1] = fmaf(s1, acc[3], z[nt][1]);
                        } else if constexpr (MODE == 2) {
                            z[nt][2] = fmaf(s0, acc[2], z[nt][2]);
                            z[nt][3] = fmaf(s1, acc[3], z[nt][3]);
                        }
                    }
                }
            }
            // ---- the values' steps; those of keys past the end may hold anything
            uint32_t vs[4][2][NG / 2];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const uint8_t *vb = ub + (nt * 8 / SB) * kSub + 2 * kCodes + kSteps;
                const int r0 = (nt * 8) % SB;
                lds<NG / 2>(vb + (r0 + key0) * NG * 2, vs[nt][0]);
                lds<NG / 2>(vb + (r0 + key1) * NG * 2, vs[nt][1]);
            }
            uint32_t seen = 0xFFFFFFFFu;  // bit nt * 2 + i (+ 8 r): row r sees key i of eight nt
            if (masked) {
                seen = 0;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int key = k0 + nt * 8 + (i ? key1 : key0);
                        if (key >= s_len) {
#pragma unroll
                            for (int h = 0; h < NG / 2; ++h) vs[nt][i][h] = 0;
                        }
#pragma unroll
                        for (int r = 0; r < NR; ++r)
                            if (key >= first[r] && key <= pos[r]) seen |= 1u << (nt * 2 + i + 8 * r);
                    }
            }
            __half2 top2 = __float2half2_rn(0.0f);
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < NG / 2; ++h)
                        top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __half2 *>(&vs[nt][i][h])));
            top2 = __hmax2(top2, __lowhigh2highlow(top2));
            uint32_t tb = *reinterpret_cast<const uint32_t *>(&top2) & 0xFFFFu;
            tb = max(tb, __shfl_xor_sync(0xFFFFFFFFu, tb, 1));
            tb = max(tb, __shfl_xor_sync(0xFFFFFFFFu, tb, 2));
            const int eb_new = max(eb, (int)(tb >> 10));

            // ---- running maximum
            float m_new[NR];
            bool moved = eb_new != eb;
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float top = m[r];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float y = z[nt][2 * r + i] * cs[r];
                        if (!(seen >> (nt * 2 + i + 8 * r) & 1)) y = -INFINITY;
                        z[nt][2 * r + i] = y;
                        top = fmaxf(top, y);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
                m_new[r] = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
                moved |= m_new[r] != m[r];
            }
            if (__any_sync(0xFFFFFFFFu, moved)) {
                const float fe = __uint_as_float((uint32_t)(127 + eb - eb_new) << 23);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float al = m_new[r] == m[r] ? 1.0f : ex2(m[r] - m_new[r]);
                    l[r] *= al;
                    const float f = al * fe;
                    m[r] = m_new[r];
#pragma unroll
                    for (int G = 0; G < NG; ++G)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            O[G][j][2 * r] *= f;
                            O[G][j][2 * r + 1] *= f;
                            if constexpr (MODE == 0) {
                                O[G][j][2] *= f;
                                O[G][j][3] *= f;
                            }
                        }
                }
                eb = eb_new;
            }
            const float pe = __uint_as_float((uint32_t)(127 + 28 - eb) << 23);  // |step| * pe < 2^14
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float mm = m[r] == -INFINITY ? 0.0f : m[r];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float e = ex2(z[nt][2 * r + i] - mm);
                        l[r] += e;
                        z[nt][2 * r + i] = e * pe;
                    }
            }

            // ---- probabilities times steps, times the values' codes
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const uint8_t *va = ub + (kk * 16 / SB) * kSub + ((kk * 16) % SB) * 16 * W;
                const uint8_t *vb = va + 8 * 16 * W;
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
                        uint32_t ah[NR][2], al[2];
#pragma unroll
                        for (int r = 0; r < NR; ++r)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int nt = 2 * kk + h;
                                const float2 d0 = unpack_f16(vs[nt][0][G / 2]), d1 = unpack_f16(vs[nt][1][G / 2]);
                                float x0 = z[nt][2 * r] * ((G & 1) ? d0.y : d0.x);
                                float x1 = z[nt][2 * r + 1] * ((G & 1) ? d1.y : d1.x);
                                if (masked) {  // a key that the row does not see may hold a step that is not finite
                                    if (!(seen >> (nt * 2 + 8 * r) & 1)) x0 = 0.0f;
                                    if (!(seen >> (nt * 2 + 1 + 8 * r) & 1)) x1 = 0.0f;
                                }
                                ah[r][h] = pack_f16(x0, x1);
                                if (MODE == 0) {
                                    const float2 b = unpack_f16(ah[r][h]);
                                    al[h] = pack_f16(x0 - b.x, x1 - b.y);
                                }
                            }
                        uint32_t y0 = __byte_perm(c00[gi / 2], c01[gi / 2], (gi & 1) ? 0x7632 : 0x5410);
                        uint32_t y1 = __byte_perm(c10[gi / 2], c11[gi / 2], (gi & 1) ? 0x7632 : 0x5410);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t mask = (j & 1) ? 0x00F000F0u : 0x000F000Fu;
                            uint32_t b0 = (y0 & mask) | 0x64006400u, b1 = (y1 & mask) | 0x64006400u;
                            __half2 &h0 = *reinterpret_cast<__half2 *>(&b0), &h1 = *reinterpret_cast<__half2 *>(&b1);
                            if (j & 1) {  // 1024 + 16 c
                                const __half2 k16 = __float2half2_rn(0.0625f), k72 = __float2half2_rn(-72.0f);
                                h0 = __hfma2(h0, k16, k72);
                                h1 = __hfma2(h1, k16, k72);
                            } else {
                                const __half2 k1032 = __float2half2_rn(-1032.0f);
                                h0 = __hadd2(h0, k1032);
                                h1 = __hadd2(h1, k1032);
                            }
                            if constexpr (MODE == 0)
                                mma_f16(O[G][j], ah[0][0], al[0], ah[0][1], al[1], b0, b1);
                            else if constexpr (MODE == 1)
                                mma_f16(O[G][j], ah[0][0], ah[0][1], b0, b1);
                            else
                                mma_f16(O[G][j], ah[0][0], ah[1][0], ah[0][1], ah[1][1], b0, b1);
                            if (j & 1) {
                                y0 >>= 8;
                                y1 >>= 8;
                            }
                        }
                    }
                }
            }
            __syncwarp();  // every lane has read the slot
            issue();
            slot = slot + 1 == kStages ? 0 : slot + 1;
            phase ^= slot == 0 ? 1u : 0u;
            step_next<R>(p, cur, lane);
        }

        // ---- the item's rows: out, or this piece's sums
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float sum = l[r];
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            const bool whole = from_start && to_end;
            const float fo = __uint_as_float((uint32_t)(127 - 28 + eb) << 23);  // undoes pe
            const float f = !whole ? fo : sum == 0.0f ? 0.0f : fo / sum;
            const int64_t rec = ((int64_t)(worker * 2 + (from_start ? 1 : 0)) * kMaxRows + g + 8 * r);
            if (live[r]) {
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a = O[G][j][2 * r], b = O[G][j][2 * r + 1];
                        if constexpr (MODE == 0) {
                            a += O[G][j][2];
                            b += O[G][j][3];
                        }
                        x[j] = a * f;
                        x[4 + j] = b * f;
                    }
                    const int el = G * 32 + t * 8;
                    if (!whole) {
                        store8<QB_T_F32>(p.part + rec * DP + el, x);
                    } else if (el < p.a.c.d) {
                        const int64_t at = otok[r] * p.a.out_stride + (int64_t)ohead[r] * p.a.c.d + el;
                        if constexpr (MODE == 0) {
                            store8<QB_T_F32>(static_cast<float *>(p.a.out) + at, x);
                        } else {
                            uint16_t *o = static_cast<uint16_t *>(p.a.out) + at;
                            if (p.a.type == QB_T_F16) store8<QB_T_F16>(o, x); else store8<QB_T_BF16>(o, x);
                        }
                    }
                }
                if (t == 0) {
                    if (!whole)
                        p.stat[rec] = make_float2(m[r], sum);
                    else if (p.a.lse)
                        p.a.lse[otok[r] * p.a.nh + ohead[r]] = (m[r] + log2f(sum)) * 0.6931471805599453f;
                }
            }
        }
        if (from_start && !to_end && lane == 0) {
            const long long item_end = end - left + item_left;  // in units of the whole work
            p.meta[worker * 2] = make_int4((int)((item_end - 1) / share), s_q0, s_T, s_kvh);
            p.meta[worker * 2 + 1] = make_int4(s_rt, 0, 0, 0);
        }
        left -= p.nosplit ? 1 : units;
    }
}

// Joins the pieces of items that lie with several workers.  Every block lists
// the items (a worker holds the start of one at most), then a warp, or the whole
// block where there are few, takes a row: the weights 2^(m_i - m) from the
// pieces' maxima, their sums added in the order of the keys.
template <int DP, int R>
__global__ void __launch_bounds__(256) kv4_combine_kernel(const StepK p) {
    constexpr int E = DP / 32;
    __shared__ int items[256 * 8];
    __shared__ int nitems, warp_n[8];
    __shared__ float red[8][DP], red_l[8];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // items in the order of the workers
    int base = 0;
    for (int i0 = 0; i0 < p.nworkers; i0 += 256) {
        const int i = i0 + threadIdx.x;
        const bool is = i < p.nworkers && p.meta[i * 2].x >= 0;
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, is);
        if (lane == 0) warp_n[warp] = __popc(b);
        __syncthreads();
        int at = base + __popc(b & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += warp_n[w];
        if (is) items[at] = i;
        for (int w = 0; w < 8; ++w) base += warp_n[w];
        __syncthreads();
    }
    if (threadIdx.x == 0) nitems = base;
    __syncthreads();
    const int tasks = nitems * R;
    const bool block_task = tasks <= (int)gridDim.x * 2;
    const int step = block_task ? gridDim.x : gridDim.x * 8;
    for (int i = block_task ? blockIdx.x : blockIdx.x * 8 + warp; i < tasks; i += step) {
        const int w0 = items[i / R], row = i % R;
        const int4 a = p.meta[w0 * 2], b = p.meta[w0 * 2 + 1];
        const int rho = b.x * R + row, j = rho / p.grp;
        if (j >= a.z) continue;  // the same for every thread of the block's task
        const int parts = a.x - w0 + 1;
        auto rec = [&](int k) { return (int64_t)((w0 + k) * 2 + (k == 0 ? 1 : 0)) * kMaxRows + row; };
        float m = -INFINITY;
        for (int k = lane; k < parts; k += 32) m = fmaxf(m, p.stat[rec(k)].x);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float mm = m == -INFINITY ? 0.0f : m;
        float acc[E], l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.0f;
        const int k0 = block_task ? warp : 0, ks = block_task ? 8 : 1;
#pragma unroll 4
        for (int k = k0; k < parts; k += ks) {
            const float2 st = p.stat[rec(k)];
            const float wgt = ex2(st.x - mm);
            l += wgt * st.y;
            const float *x = p.part + rec(k) * DP + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(x + e);
                acc[e] += wgt * v.x;
                acc[e + 1] += wgt * v.y;
            }
        }
        if (block_task) {
            __syncthreads();  // red of the task before has been read
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
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t tok = a.y + j;
        const int head = a.w * p.grp + rho - j * p.grp;
        const int64_t at = tok * p.a.out_stride + (int64_t)head * p.a.c.d;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int el = lane * E + e;
            const float y = acc[e] * inv;
            if (el < p.a.c.d) {
                if (p.a.type == QB_T_F32) static_cast<float *>(p.a.out)[at + el] = y;
                else if (p.a.type == QB_T_F16) static_cast<__half *>(p.a.out)[at + el] = __float2half_rn(y);
                else static_cast<__nv_bfloat16 *>(p.a.out)[at + el] = __float2bfloat16_rn(y);
            }
        }
        if (lane == 0 && p.a.lse) p.a.lse[tok * p.a.nh + head] = (m + log2f(l)) * 0.6931471805599453f;
    }
}

// ---------------------------------------------------------------- launch

// an item of at most this many keys is not split (and no join is launched)
constexpr int kNoSplitKeys = 256;

template <int DP, int MODE, int SB>
static int launch_step_k(StepK &p, int grid, cudaStream_t stream) {
    constexpr int smem = kStepWarps * step_stages<DP>() * step_unit_bytes<DP>();
    auto *f = kv4_step_kernel<DP, MODE, SB>;
    if (ensure_smem_limit(reinterpret_cast<const void *>(f), smem) != QB_OK) return QB_E_CUDA;
    if (const int rc = launch_pdl(f, dim3((unsigned)grid), dim3(kStepWarps * 32), smem, stream, p)) return rc;
    if (p.nosplit) return QB_OK;
    return launch_pdl(kv4_combine_kernel<DP, step_rows<MODE>()>, dim3((unsigned)grid), dim3(256), 0, stream, p);
}

template <int DP, int MODE>
static int launch_step_m(StepK &p, int grid, cudaStream_t stream) {
    return p.a.c.page == 16 ? launch_step_k<DP, MODE, 16>(p, grid, stream)
                            : launch_step_k<DP, MODE, 32>(p, grid, stream);
}

template <int DP>
int launch_kv4_step(const Kv4AttnArgs &a, cudaStream_t stream) {
    StepK p = {};
    p.a = a;
    p.grp = a.nh / a.c.nkv;
    const int grid = std::min(num_sms(), 256);
    p.nworkers = grid * kStepWarps;
    p.min_share = 4;
    p.nosplit = (int64_t)a.s.maxp * a.c.page <= kNoSplitKeys;
    p.part = reinterpret_cast<float *>(a.ws);
    p.stat = reinterpret_cast<float2 *>(p.part + (int64_t)p.nworkers * 2 * kMaxRows * DP);
    p.meta = reinterpret_cast<int4 *>(p.stat + (int64_t)p.nworkers * 2 * kMaxRows);
    if (a.type == QB_T_F32) return launch_step_m<DP, 0>(p, grid, stream);
    // rows a sequence and key head, on average
    if (a.ntok * p.grp <= (int64_t)8 * a.s.nseq) return launch_step_m<DP, 1>(p, grid, stream);
    return launch_step_m<DP, 2>(p, grid, stream);
}

int launch_kv4_step_64(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_128(const Kv4AttnArgs &a, cudaStream_t stream);
int launch_kv4_step_256(const Kv4AttnArgs &a, cudaStream_t stream);

}  // namespace qb
