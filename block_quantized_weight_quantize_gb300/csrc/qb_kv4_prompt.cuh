// qb_kv4_prompt.cuh -- attention of many new tokens a sequence (prompts and
// their chunks) over the paged 4-bit cache, in half precision, on the
// fifth-generation tensor cores.
//
// Mathematics: as in qb_kv4_step.cuh, but with 128 rows and more a key head the
// products bound it, so keys and values are decoded once a tile to f16
// ((code - 8) * step, rounded once) and the tensor cores do the rest:
//     S = Q K^T (f32), P = 2^(S cs - m) (f16), O += P V (f32),
// m a running maximum that moves only when it has to rise by more than 8 (the
// factor 2^8 fits f16), when O is rescaled in tensor memory; sums in f32.
//
// Work: an item is 256 rows (two tiles of 128; row = token * heads of the key
// head + head) of one sequence and key head; a block takes items, the longest
// first.  Roles of a block's 16 warps:
//   0-3, 4-7  softmax of tile 0, 1: a thread a row, 32 scores at a time from
//             tensor memory, P back over the scores
//   8-11      decoders: a thread a key, rows loaded a tile ahead into
//             registers, f16 core matrices (8 rows of 16 bytes) to shared memory
//   12        issues the products: PV0(i), S0(i+1), then PV1(i), S1(i+1), so that
//             one tile's softmax runs under the other tile's products
// (Registers: 152 a softmax thread, 104 another's.)
// Core matrices: K [dims/8][128 keys][8 dims] (K-major), V the same (dims along
// N: MN-major), Q like K; the order of dims within and of groups of eight is the one
// that unpacking gives, and is undone in Q's rows and the output's columns.
//
// Values out of the ordinary: a key whose steps reach 2^12 is decoded 2^-4
// smaller, and its scores or probabilities multiplied by 16; a group whose step
// is not finite is decoded as zeros and marks the rows that see it, whose
// outputs of that group are NaN.
#pragma once

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
};

struct PromptItem {
    int row, len, T, q0, kvh, rp;
    int t0, n;  // first key tile, tiles
};

template <int DP>
struct PromptSmem {
    static constexpr int kTileBytes = kPromptTile * DP * 2;
    alignas(128) uint8_t q[kPromptQ][kTileBytes];
    alignas(128) uint8_t k[2][kTileBytes];
    alignas(128) uint8_t v[2][kTileBytes];
    uint16_t flags[4][kPromptTile];  // of a tile's keys: 1 K, 2 V decoded 2^-4 smaller; from bit 8 the groups that are not finite
    uint32_t any[4][4];              // whether a decoder warp's keys have one
    uint64_t q_full[kPromptQ], s_full[kPromptQ], p_ready[kPromptQ], o_done[kPromptQ];
    uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
    uint32_t tmem;
    int chunk_sum[8192 / 32 + 1];
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
    for (int i = 0; i < 4; ++i) o[i] = prompt_half2(__hmul2(*reinterpret_cast<const __half2 *>(&b[i]), step));
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The whole warp's wait: false (for all of it) if any lane's ran out.
__device__ __forceinline__ bool prompt_wait(uint64_t *bar, uint32_t parity, int *fault) {
    const bool ok = mbar_try_wait(bar, parity) || mbar_wait_sleep(bar, parity, fault);
    return __all_sync(0xFFFFFFFFu, ok);
}

// The groups that are not finite among the keys lo..hi of a step.
static __device__ __noinline__ uint32_t prompt_bad(const uint16_t *flags, int lo, int hi) {
    uint32_t bad = 0;
    for (int i = max(lo, 0); i <= min(hi, kPromptTile - 1); ++i) bad |= flags[i] >> 8;
    return bad;
}

// What a row's softmax carries from tile to tile.
struct PromptRow {
    float cs, m, l;   // factor of the scores, running maximum, sum
    int lo, hi;       // columns lo..hi of the step are seen
};

// The maximum rises to mn in lanes where that is more than m: O (DP columns, if
// any products were added), the `done` columns of this step's probabilities and the sum shrink.
template <int DP>
static __device__ __noinline__ bool prompt_rescale(uint32_t tS, uint32_t tO, int done, float &m, float &l, float mn,
                                                   bool have_o, uint64_t *o_done, uint32_t parity, int *fault) {
    const float al = mn == m ? 1.0f : prompt_ex2(m - mn);
    l *= al;
    m = mn;
    if (have_o) {
        if (!prompt_wait(o_done, parity, fault)) return false;
        tc_fence_after();
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
        const __half2 a2 = __float2half2_rn(al);
        for (int c = 0; c < done; c += 32) {  // 16 or 48 columns: the rest of the last 32 is scores, kept
            uint32_t o[32];
            tc_ld32(tS + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < done) o[i] = prompt_half2(__hmul2(*reinterpret_cast<const __half2 *>(&o[i]), a2));
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

// A step's row: 64 scores in tensor memory, 32 at a time (the next ones on
// their way), become probabilities 2^(s cs - m) as f16 over them (32 scores'
// columns have been read when the 16 columns of their probabilities are
// written).  MASKED: scores outside columns lo..hi count as -infinity; ODD:
// flagged keys' scores or probabilities are 16 times larger.
template <int DP, bool MASKED, bool ODD>
__device__ __forceinline__ bool prompt_step(uint32_t tS, uint32_t tO, PromptRow &row, const uint16_t *flags, bool have_o,
                                            uint64_t *o_done, uint32_t parity, int *fault) {
    uint32_t s[2][32];
    const uint64_t cs2 = pair_f32(row.cs, row.cs);
    uint64_t sum = 0;  // (0, 0)
    bool ok = true;
    tc_ld32_begin(tS, s[0]);
#pragma unroll
    for (int c = 0; c < kPromptTile / 32; ++c) {
        uint32_t (&x)[32] = s[c & 1];
        tc_ld_wait(x);
        if (c + 1 < kPromptTile / 32) tc_ld32_begin(tS + 32 * (c + 1), s[(c + 1) & 1]);
        if (ODD || MASKED) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                if (ODD && (flags[32 * c + i] & 1)) x[i] = __float_as_uint(__uint_as_float(x[i]) * 16.0f);
                if (32 * c + i > row.hi || 32 * c + i < row.lo) x[i] = 0xFF800000u;
            }
        }
        float t0 = __uint_as_float(x[0]), t1 = __uint_as_float(x[1]);
#pragma unroll
        for (int i = 2; i < 32; i += 2) {
            t0 = fmaxf(t0, __uint_as_float(x[i]));
            t1 = fmaxf(t1, __uint_as_float(x[i + 1]));
        }
        const float z = fmaxf(t0, t1) * row.cs;
        if (__any_sync(0xFFFFFFFFu, z > row.m + 8.0f)) {
            if (c + 1 < kPromptTile / 32) tc_ld_wait(s[(c + 1) & 1]);
            const float2 part = unpair_f32(sum);
            float l = row.l + (part.x + part.y), m = row.m;
            sum = 0;
            ok = prompt_rescale<DP>(tS, tO, 16 * c, m, l, z > m + 8.0f ? z : m, have_o, o_done, parity, fault) && ok;
            row.l = l;
            row.m = m;
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
    }
    const float2 part = unpair_f32(sum);
    row.l += part.x + part.y;
    return ok;
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
        fence_mbar_init();
    }
    if (warp == 12) {
        tc_alloc(&sm.tmem, 512);
        tc_relinquish();
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- the items: an item's number counts sequences, row pairs, key heads
    const int nseq = p.a.s.nseq, nchunks = (nseq + 31) / 32;
    auto info = [&](int s, bool report) {
        SeqInfo r = {0, 0, 0, 0};
        if (s < nseq) r = seq_info(p.a, s, report);
        return r;
    };
    auto row_pairs = [&](int T) { return (T * p.grp + kPromptRows - 1) / kPromptRows; };
    for (int c = warp; c < nchunks; c += kPromptThreads / 32) {
        int n = p.a.c.nkv * row_pairs(info(c * 32 + lane, blockIdx.x == 0).T);
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
        if (lane == 0) sm.chunk_sum[c] = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) {
        int sum = 0;
        for (int c = 0; c < nchunks; ++c) {
            const int n = sm.chunk_sum[c];
            sm.chunk_sum[c] = sum;
            sum += n;
        }
        sm.chunk_sum[nchunks] = sum;
    }
    __syncthreads();
    const int total = sm.chunk_sum[nchunks];
    const uint32_t tb = sm.tmem;
    // this block's k-th item, the longest first (a sequence's last rows see the most keys), to and fro
    auto item_at = [&](int k, PromptItem &it) {
        const int64_t x = (int64_t)k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if (x >= total) return false;
        const int idx = total - 1 - (int)x;
        int lo = 0, hi = nchunks;
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (sm.chunk_sum[m] <= idx) lo = m; else hi = m;
        }
        const SeqInfo q = info(lo * 32 + lane, false);
        const int n = p.a.c.nkv * row_pairs(q.T);
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += y;
        }
        const int before = sm.chunk_sum[lo] + sum - n;
        const uint32_t ok = __ballot_sync(0xFFFFFFFFu, n > 0 && before <= idx);
        const int l = 31 - __clz(ok);
        const int rem = idx - __shfl_sync(0xFFFFFFFFu, before, l);
        it.row = __shfl_sync(0xFFFFFFFFu, q.row, l);
        it.len = __shfl_sync(0xFFFFFFFFu, q.len, l);
        it.T = __shfl_sync(0xFFFFFFFFu, q.T, l);
        it.q0 = __shfl_sync(0xFFFFFFFFu, q.q0, l);
        it.rp = rem / p.a.c.nkv;
        it.kvh = rem - it.rp * p.a.c.nkv;
        const int j_lo = it.rp * kPromptRows / p.grp, j_hi = min(it.T - 1, (it.rp * kPromptRows + kPromptRows - 1) / p.grp);
        const int pos_lo = it.len - it.T + j_lo, pos_hi = it.len - it.T + j_hi;
        const int first = p.a.window ? max(0, pos_lo - p.a.window + 1) : 0;
        it.t0 = first / kPromptTile;
        it.n = pos_hi < 0 ? 0 : pos_hi / kPromptTile + 1 - it.t0;
        return true;
    };

    PromptItem it;
    // 128 registers a thread of 4 warpgroups at launch: 152 + 152 + 104 + 104 = 4 * 128
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 152;");
        // ================================================= softmax
        const int q = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tb + lanes + 128u * q, tO = tb + lanes + 256u + (uint32_t)DP * q;
        uint32_t tiles = 0;  // of this row tile so far
        bool ok = true;
        for (int k = 0; ok && item_at(k, it); ++k) {
            const int rho = it.rp * kPromptRows + q * kPromptTile + r, j = rho / p.grp;
            const bool live = j < it.T;
            const int pos = live ? it.len - it.T + j : -1;
            const int first = p.a.window ? max(0, pos - p.a.window + 1) : 0;
            const int64_t tok = it.q0 + j;
            const int head = it.kvh * p.grp + rho - j * p.grp;
            float cs = 0.0f;
            if (it.n > 0) {
                // the row's queries as f16, its largest magnitude scaled into [2^14, 2^15)
                const uint16_t *src = static_cast<const uint16_t *>(p.a.q) + tok * p.a.q_stride + (int64_t)head * p.a.c.d;
                auto load = [&](int o, float (&x)[8]) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = 0.0f;
                    if (!live || o * 8 >= p.a.c.d) return;
                    if (p.a.type == QB_T_F16) load8<QB_T_F16>(src + o * 8, x); else load8<QB_T_BF16>(src + o * 8, x);
                };
                float top = 0.0f;
#pragma unroll 4
                for (int o = 0; o < DP / 8; ++o) {
                    float x[8];
                    load(o, x);
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
                }
                const int e = top > 0.0f ? max((int)(__float_as_uint(top) >> 23) - 127, -100) : 8;
                const float f = copysignf(__uint_as_float((uint32_t)(127 + 8 - e) << 23), p.a.scale);
                // not zero, so that a score that is masked stays -inf
                cs = fmaxf(fabsf(p.a.scale) * 1.4426950408889634f * exp2f((float)(e - 8)), 1e-37f);
                uint8_t *dst = sm.q[q] + r * 16;
#pragma unroll 4
                for (int o = 0; o < DP / 8; ++o) {
                    float x[8];
                    load(o, x);
                    uint4 u;
                    u.x = prompt_half2(__floats2half2_rn(x[0] * f, x[4] * f));
                    u.y = prompt_half2(__floats2half2_rn(x[1] * f, x[5] * f));
                    u.z = prompt_half2(__floats2half2_rn(x[2] * f, x[6] * f));
                    u.w = prompt_half2(__floats2half2_rn(x[3] * f, x[7] * f));
                    *reinterpret_cast<uint4 *>(dst + o * kOctStride) = u;
                }
                fence_async_shared();
                mbar_arrive(&sm.q_full[q]);
            }
            // tiles whose keys all of this row tile's rows see need no mask
            const int j_lo = (it.rp * kPromptRows + q * kPromptTile) / p.grp;
            const int j_hi = min(it.T - 1, (it.rp * kPromptRows + q * kPromptTile + kPromptTile - 1) / p.grp);
            const int pos_lo = j_lo < it.T ? it.len - it.T + j_lo : -1;
            const int first_hi = p.a.window ? max(0, it.len - it.T + j_hi - p.a.window + 1) : 0;
            PromptRow row = {cs, -INFINITY, 0.0f, 0, 0};
            uint32_t bad = 0;
            for (int i = 0; i < it.n; ++i, ++tiles) {
                const int k0 = (it.t0 + i) * kPromptTile;
                if (!(ok = prompt_wait(&sm.s_full[q], tiles & 1, p.a.fault))) break;
                tc_fence_after();
                const uint32_t sl = tiles & 3, par = (tiles - 1) & 1;
                const bool odd = (sm.any[sl][0] | sm.any[sl][1] | sm.any[sl][2] | sm.any[sl][3]) != 0;
                const bool masked = k0 + kPromptTile - 1 > pos_lo || k0 < first_hi;
                const uint16_t *flags = sm.flags[sl];
                row.hi = pos - k0;
                row.lo = first - k0;
                if (odd) {
                    bad |= prompt_bad(flags, row.lo, row.hi);
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
            if (it.n > 0) {
                if (!(ok = prompt_wait(&sm.o_done[q], (tiles - 1) & 1, p.a.fault))) break;
                tc_fence_after();
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *out = static_cast<uint16_t *>(p.a.out) + tok * p.a.out_stride + (int64_t)head * p.a.c.d;
            // 32 columns are chunks 2kk, 2kk + 1 (W = 4; all four of W = 2's eight dims): eight dims of every group
#pragma unroll
            for (int kk = 0; kk < DP / 32; ++kk) {
                uint32_t o[32];
                __syncwarp();
                if (it.n > 0) {
                    tc_ld32(tO + 32 * kk, o);
                } else {
#pragma unroll
                    for (int i2 = 0; i2 < 32; ++i2) o[i2] = 0u;
                }
                // column (c * (W / 2) + u) * 8 + 2 j + h is dim (2 u + h) * 32 + 4 c + j
                constexpr int CPL = 8 / W;  // chunks in 32 columns
                if (live) {
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
                        const int el = G * 32 + kk * 4 * CPL;
#pragma unroll
                        for (int h = 0; h < 4 * CPL; h += 8) {
                            if (el + h >= p.a.c.d) continue;
                            const float (&y)[8] = *reinterpret_cast<const float (*)[8]>(&x[h]);
                            if (p.a.type == QB_T_F16) store8<QB_T_F16>(out + el + h, y); else store8<QB_T_BF16>(out + el + h, y);
                        }
                    }
                }
            }
            if (live && p.a.lse) p.a.lse[tok * p.a.nh + head] = (m + log2f(l)) * 0.6931471805599453f;
            __syncwarp();
            tc_fence_before();  // the reads of O, before the next item's products
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        // ================================================= decoders: a thread a key
        const CentreK ck;
        const int r = threadIdx.x - 8 * 32, dw = warp - 8;
        const int page = p.a.c.page, code_bytes = page * DP / 2, step_bytes = page * DP / 16;
        uint32_t kt = 0;
        bool ok = true;
        constexpr int NV = DP / 32;  // 16-byte pieces of a row's codes
        uint4 kx[NV], vx[NV];
        uint32_t ks[NG / 2], vs[NG / 2];
        for (int k = 0; ok && item_at(k, it); ++k) {
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
            if (it.n > 0) load(it.t0, kx, ks, vx, vs);
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
                if (!(ok = prompt_wait(&sm.k_free[slot], ph ^ 1u, p.a.fault))) break;
                // the tile's flags: three tiles at most are in use, four are held
                sm.flags[kt & 3][r] = (uint16_t)fl;
                const uint32_t any = __ballot_sync(0xFFFFFFFFu, fl != 0);
                if (lane == 0) sm.any[kt & 3][dw] = any;
                uint8_t *dst = sm.k[slot] + r * 16;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int gi = 0; gi < W; ++gi) {
                        const int wi = t * W + gi;  // the row's word: elements 8 t .. of group gi
                        const uint4 &u = kc[wi / 4];
                        const uint32_t w = wi % 4 == 0 ? u.x : wi % 4 == 1 ? u.y : wi % 4 == 2 ? u.z : u.w;
                        const __half2 sp = *reinterpret_cast<const __half2 *>(&kst[gi / 2]);
                        *reinterpret_cast<uint4 *>(dst + (gi * 4 + t) * kOctStride) =
                            prompt_decode(ck, w, (gi & 1) ? __high2half2(sp) : __low2half2(sp));
                    }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.k_full[slot]);
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
        uint32_t kt = 0, items = 0;  // key tiles, items so far
        bool ok = warp == 12;
        // S = Q K^T with key tile t
        auto scores = [&](int q, uint32_t t) {
            const uint32_t qa = smem_u32(sm.q[q]), ka = smem_u32(sm.k[t & 1]);
            if (elect_one()) {
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    tc_mma_ss(tb + 128u * q, tc_desc(qa + 2 * s * kOctStride, kOctStride, 128),
                              tc_desc(ka + 2 * s * kOctStride, kOctStride, 128), idS, s != 0);
                tc_commit(&sm.s_full[q]);
                if (q == kPromptQ - 1) tc_commit(&sm.k_free[t & 1]);
            }
            __syncwarp();
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
        for (int k = 0; ok && item_at(k, it); ++k) {
            if (it.n == 0) continue;
            for (int q = 0; q < kPromptQ && ok; ++q) ok = prompt_wait(&sm.q_full[q], items & 1, p.a.fault);
            ++items;
            if (!ok || !(ok = prompt_wait(&sm.k_full[kt & 1], (kt >> 1) & 1, p.a.fault))) break;
            tc_fence_after();
            for (int q = 0; q < kPromptQ; ++q) scores(q, kt);
            for (int i = 0; ok && i < it.n; ++i, ++kt) {
                const bool more = i + 1 < it.n;
                if (!(ok = prompt_wait(&sm.v_full[kt & 1], (kt >> 1) & 1, p.a.fault))) break;
                if (more && !(ok = prompt_wait(&sm.k_full[(kt + 1) & 1], ((kt + 1) >> 1) & 1, p.a.fault))) break;
                for (int q = 0; q < kPromptQ; ++q) {
                    if (!(ok = prompt_wait(&sm.p_ready[q], kt & 1, p.a.fault))) break;
                    tc_fence_after();
                    outputs(q, kt, i == 0);
                    if (!more) continue;
                    // products with different accumulators are not ordered: the next scores,
                    // which go where P is, wait until it has been read
                    if (!(ok = prompt_wait(&sm.o_done[q], kt & 1, p.a.fault))) break;
                    tc_fence_after();
                    scores(q, kt + 1);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 12) tc_dealloc(tb, 512);
}

template <int DP>
int launch_kv4_prompt(const Kv4AttnArgs &a, cudaStream_t stream) {
    PromptK p;
    p.a = a;
    p.grp = a.nh / a.c.nkv;
    constexpr int smem = (int)sizeof(PromptSmem<DP>) + 128;
    auto *f = kv4_prompt_kernel<DP>;
    if (ensure_smem_limit(reinterpret_cast<const void *>(f), smem) != QB_OK) return QB_E_CUDA;
    return launch_pdl(f, dim3((unsigned)num_sms()), dim3(kPromptThreads), smem, stream, p);
}

}  // namespace qb

