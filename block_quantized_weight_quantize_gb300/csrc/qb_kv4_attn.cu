// qb_kv4_attn.cu -- attention over the paged 4-bit cache (qgemv.h: kv4_attn).
//
// One warp per (token, query head): 32 keys a turn, a lane a key for the
// scores, then every lane its share of the output's elements; the softmax's
// maximum and sum run along the keys.
#include <cstdint>

#include "qb_kv4.cuh"

namespace qb {

template <int TYPE, int DP>
__global__ void __launch_bounds__(256) kv4_attn_simple_kernel(const Kv4AttnArgs p) {
    constexpr int kOcts = DP / 8, kPer = DP / 32, kW = DP / 32 < 4 ? DP / 32 : 4;
    __shared__ float qs[8][DP];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 8 + warp;
    if (item >= p.ntok * p.nh) return;
    const int64_t tok = item / p.nh;
    const int h = (int)(item - tok * p.nh), kvh = h / (p.nh / p.c.nkv);
    // the token's sequence: the last one that starts at or before it
    int s = (int)tok, T = 1, j = 0;
    if (p.s.q_start) {
        int lo = 0, hi = p.s.nseq;
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (p.s.q_start[m] <= tok) lo = m; else hi = m;
        }
        s = lo;
        T = p.s.q_start[s + 1] - p.s.q_start[s];
        j = (int)(tok - p.s.q_start[s]);
        if (j < 0 || j >= T) return;
    }
    const int row = p.s.rows ? p.s.rows[s] : s;
    int len = 0;
    if (row < 0 || row >= p.s.nrows) {
        if (lane == 0) atomicOr(p.fault, kFaultIndex);
    } else {
        len = (int)min((int64_t)max(p.s.lens[row], 0), (int64_t)p.s.maxp * p.c.page);
    }
    const int pos = len - T + j;
    const int first = p.window ? max(0, pos - p.window + 1) : 0;
    const int32_t *tab = p.s.tables + (int64_t)row * p.s.maxp;
    for (int o = lane; o < kOcts; o += 32) {
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (o * 8 < p.c.d)
            load8<TYPE>(static_cast<const uint8_t *>(p.q) +
                            (tok * p.q_stride + (int64_t)h * p.c.d + o * 8) * type_bytes(TYPE),
                        x);
        for (int i = 0; i < 8; ++i) qs[warp][o * 8 + i] = x[i];
    }
    __syncwarp();
    float m = -INFINITY, l = 0.0f, acc[kPer];
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    const int page = p.c.page, code_bytes = page * DP / 2, step_bytes = page * DP / 16;
    for (int k0 = first & ~31; k0 <= pos; k0 += 32) {
        const int key = k0 + lane;
        const bool seen = key >= first && key <= pos;
        const uint8_t *b = p.c.data;
        const int r = key & (page - 1);
        float z = -INFINITY;
        if (seen) {
            int pg = tab[key >> p.c.pshift];
            if (pg < 0 || pg >= p.c.npages) {
                atomicOr(p.fault, kFaultIndex);
                pg = 0;
            }
            b += ((int64_t)pg * p.c.nkv + kvh) * p.c.block_bytes;
            z = 0.0f;
            for (int g = 0; g < DP / 32; ++g) {
                const float st = __half2float(*reinterpret_cast<const __half *>(b + code_bytes + (r * (DP / 32) + g) * 2));
                float dot = 0.0f;
                for (int o = 4 * g; o < 4 * g + 4; ++o) {
                    const uint32_t w = *reinterpret_cast<const uint32_t *>(b + kv4_key_word(page, kW, r, o));
                    for (int i = 0; i < 8; ++i) dot += qs[warp][o * 8 + i] * (float)((int)((w >> (4 * i)) & 15) - 8);
                }
                z += dot * st;
            }
            z *= p.scale;
        }
        float top = z;
        bool nan = z != z;
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const float mn = fmaxf(m, top), safe = mn == -INFINITY ? 0.0f : mn;
        const float a = expf(m - safe), e = expf(z - safe);
        l = l * a + e;
        for (int i = 0; i < kPer; ++i) acc[i] *= a;
        m = mn;
        const unsigned long long bp = reinterpret_cast<unsigned long long>(b);
        for (int k = 0; k < 32; ++k) {
            const float ek = __shfl_sync(0xFFFFFFFFu, e, k);
            const uint8_t *bk = reinterpret_cast<const uint8_t *>(__shfl_sync(0xFFFFFFFFu, bp, k));
            if (!__shfl_sync(0xFFFFFFFFu, (int)seen, k)) continue;
            const int rk = (k0 + k) & (page - 1);
            const uint8_t *v = bk + code_bytes + step_bytes;
            for (int i = 0; i < kPer; ++i) {
                const int el = lane * kPer + i, o = el / 8;
                const uint32_t hw = *reinterpret_cast<const uint16_t *>(v + kv4_value_half(page, kW, rk, o, (el & 7) / 4));
                const float st = __half2float(*reinterpret_cast<const __half *>(v + code_bytes + (rk * (DP / 32) + el / 32) * 2));
                acc[i] += ek * ((float)((int)((hw >> (4 * (el & 3))) & 15) - 8) * st);
            }
        }
        (void)nan;
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    __syncwarp();
    for (int i = 0; i < kPer; ++i) qs[warp][lane * kPer + i] = acc[i] * inv;
    __syncwarp();
    for (int o = lane; o < kOcts; o += 32)
        if (o * 8 < p.c.d) {
            float x[8];
            for (int i = 0; i < 8; ++i) x[i] = qs[warp][o * 8 + i];
            store8<TYPE>(static_cast<uint8_t *>(p.out) +
                             (tok * p.out_stride + (int64_t)h * p.c.d + o * 8) * type_bytes(TYPE),
                         x);
        }
    if (lane == 0 && p.lse) p.lse[tok * p.nh + h] = m + logf(l);
}

int64_t kv4_attn_ws(int, int, int) { return 16; }

template <int TYPE>
static int launch_simple(const Kv4AttnArgs &a, cudaStream_t stream) {
    auto *f = a.c.dp == 64 ? kv4_attn_simple_kernel<TYPE, 64>
              : a.c.dp == 128 ? kv4_attn_simple_kernel<TYPE, 128> : kv4_attn_simple_kernel<TYPE, 256>;
    return launch_pdl(f, dim3((unsigned)((a.ntok * a.nh + 7) / 8)), dim3(256), 0, stream, a);
}

int launch_kv4_attn(const Kv4AttnArgs &a, cudaStream_t stream) {
    return a.type == QB_T_F32 ? launch_simple<QB_T_F32>(a, stream)
           : a.type == QB_T_F16 ? launch_simple<QB_T_F16>(a, stream) : launch_simple<QB_T_BF16>(a, stream);
}

}  // namespace qb
