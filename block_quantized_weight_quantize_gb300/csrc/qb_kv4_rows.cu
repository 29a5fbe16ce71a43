// qb_kv4_rows.cu -- rows into and out of the paged 4-bit cache (qgemv.h:
// kv4_append, kv4_read).
//
// A thread takes 16 consecutive elements of a row: two words of a key row, four
// halves of a value row; two neighbouring threads hold a group of 32 and find
// its step by a shuffle.  A block has one side (keys, values) of one key head,
// and a thread two tokens' rows, whose loads are under way before the first is
// used.  Each element is read once and its half byte written once (or the
// reverse); instructions bound it, so that there is no conversion a code (with
// 1.5 * 2^23 + 8 added, an element over its step has its code in its low bits,
// rounded to nearest even by the addition, and eight of them join by shifted
// additions) and f32 goes two at a time.  Measured on 20011 tokens of 8 heads of
// 128 in bf16 (105 MB each way): append 28 us (3.7 TB/s), read 24 us (4.4 TB/s); 8 elements a thread took 39 and 31 us.
#include <cstdint>

#include "qb_kv4.cuh"

namespace qb {

struct RowsK {
    Kv4View c;
    const void *src[2];
    void *dst[2];
    int64_t stride[2];
    const int32_t *slots;
    int64_t n;
    int *fault;
};

constexpr int kRowsThreads = 256;
constexpr int kRows = 2;  // tokens a thread

// The thread's 16 elements of a row, its first token and the distance to its
// next; byte offsets in a block's side: of its first key word (the second is 4 w
// further) or value half (the others 2 w further each, and all by `turn` in the
// rows whose halves are exchanged).
struct RowPlace {
    int64_t token;
    int el, step, off, turn, w;
};
__device__ __forceinline__ RowPlace row_place(const RowsK &p, int side) {
    const int sh = p.c.dp == 64 ? 2 : p.c.dp == 128 ? 3 : 4;  // threads a row: 2^sh
    RowPlace r;
    const int i = threadIdx.x & ((1 << sh) - 1), G = i >> 1, t = 2 * (i & 1);
    r.el = 16 * i;
    r.step = kRowsThreads >> sh;
    r.token = (int64_t)blockIdx.x * r.step * kRows + (threadIdx.x >> sh);
    r.w = min(p.c.dp / 32, 4);
    const int plane = (G >> 2) * p.c.page * 16 * r.w;
    r.off = plane + (side ? 2 * t * r.w + (G & 3) : 2 * (t * r.w + (G & 3))) * 2;
    r.turn = t ? -8 * r.w : 8 * r.w;
    return r;
}

// A token's slot, or -1: none, or past the cache (reported).
__device__ __forceinline__ int row_slot(const RowsK &p, int64_t token) {
    if (token >= p.n) return -1;
    const int slot = p.slots[token];
    if ((slot >> p.c.pshift) < p.c.npages) return slot;
    atomicOr(p.fault, kFaultIndex);
    return -1;
}

// The block of a slot's page and head, at its keys or values.
__device__ __forceinline__ uint8_t *row_block(const RowsK &p, int slot, int head, int side) {
    const int area = p.c.page * p.c.dp / 2 + p.c.page * p.c.dp / 16;
    return p.c.data + ((int64_t)(slot >> p.c.pshift) * p.c.nkv + head) * p.c.block_bytes + (side ? area : 0);
}

// Eight elements' codes under the step s (its reciprocal inv; 0: all zeros) as a word.
__device__ __forceinline__ uint32_t row_word(const float *x, float s, float inv) {
    constexpr uint32_t kMagic = 0x4B400008u;  // 1.5 * 2^23 + 8: its last place is 1
    uint32_t word = 0, base = 0;
    const uint64_t inv2 = pair_f32(inv, inv), magic2 = pair_f32(__uint_as_float(kMagic), __uint_as_float(kMagic));
    uint64_t odd2 = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t y2 = mul_f32x2(pair_f32(x[i], x[i + 1]), inv2);
        odd2 = fma_f32x2(y2, 0, odd2);
        const float2 y = unpair_f32(y2);
        const float2 c = unpair_f32(add_f32x2(pair_f32(fminf(y.x, 7.0f), fminf(y.y, 7.0f)), magic2));
        word += __float_as_uint(c.x) << (4 * i);  // 0x4B400000 + code
        word += __float_as_uint(c.y) << (4 * i + 4);
        base += (0x4B400000u << (4 * i)) + (0x4B400000u << (4 * i + 4));
    }
    word -= base;
    // An element over its step lies in -8 .. 8 but for what the step's rounding adds,
    // half a place at most where the step is normal.  Else, and where a product is
    // not finite (NaN stands for zero), one at a time:
    const float2 odd = unpair_f32(odd2);
    if (odd.x + odd.y != 0.0f || (fabsf(s) < 6.104e-5f && s != 0.0f)) {
        word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = __fmul_rn(x[i], inv);
            word |= (uint32_t)(y == y ? 8 + (int)rintf(fminf(fmaxf(y, -8.0f), 7.0f)) : 8) << (4 * i);
        }
    }
    return word;
}

template <int TYPE>
__global__ void __launch_bounds__(kRowsThreads) kv4_append_kernel(const RowsK p) {
    pdl_launch_dependents();
    pdl_wait();
    const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
    const RowPlace r = row_place(p, side);
    const int code_bytes = p.c.page * p.c.dp / 2;
    const int64_t stride = side ? p.stride[1] : p.stride[0];
    const uint8_t *src = static_cast<const uint8_t *>(side ? p.src[1] : p.src[0]) +
                         (r.token * stride + (int64_t)head * p.c.d + r.el) * type_bytes(TYPE);
    float x[kRows][16];
    int slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        slot[k] = row_slot(p, r.token + k * r.step);
        const bool there = r.token + k * r.step < p.n;
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            float (&y)[8] = *reinterpret_cast<float (*)[8]>(&x[k][h]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = 0.0f;
            if (there && r.el + h < p.c.d) load8<TYPE>(src + (k * r.step * stride + h) * type_bytes(TYPE), y);
        }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        // the group's extremes: fmaxf and fminf pass NaN over
        float hi = 0.0f, lo = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            hi = fmaxf(hi, x[k][i]);
            lo = fminf(lo, x[k][i]);
        }
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, 1));
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, 1));
        const __half step = __float2half_rn((hi >= -lo ? hi : lo) * -0.125f);
        const float s = __half2float(step);
        const float inv = s == 0.0f ? 0.0f : __frcp_rn(s);
        const uint32_t w0 = row_word(x[k], s, inv), w1 = row_word(x[k] + 8, s, inv);
        if (slot[k] < 0) continue;
        uint8_t *b = row_block(p, slot[k], head, side);
        const int row = slot[k] & (p.c.page - 1);
        uint8_t *c = b + r.off + row * 16 * r.w;
        if (side == 0) {
            *reinterpret_cast<uint32_t *>(c) = w0;
            *reinterpret_cast<uint32_t *>(c + 4 * r.w) = w1;
        } else {
            if (row & 2) c += r.turn;
            *reinterpret_cast<uint16_t *>(c) = (uint16_t)w0;
            *reinterpret_cast<uint16_t *>(c + 2 * r.w) = (uint16_t)(w0 >> 16);
            *reinterpret_cast<uint16_t *>(c + 4 * r.w) = (uint16_t)w1;
            *reinterpret_cast<uint16_t *>(c + 6 * r.w) = (uint16_t)(w1 >> 16);
        }
        if ((r.el & 16) == 0) *reinterpret_cast<__half *>(b + code_bytes + (row * (p.c.dp / 32) + (r.el >> 5)) * 2) = step;
    }
}

template <int TYPE>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(const RowsK p) {
    pdl_launch_dependents();
    pdl_wait();
    const int head = blockIdx.y >> 1, side = blockIdx.y & 1;
    const RowPlace r = row_place(p, side);
    const int code_bytes = p.c.page * p.c.dp / 2;
    if (r.el >= p.c.d) return;
    int slot[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) slot[k] = row_slot(p, r.token + k * r.step);
    uint32_t word[kRows][2];
    float s[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        word[k][0] = word[k][1] = 0x88888888u;  // zeros
        s[k] = 0.0f;
        if (slot[k] < 0) continue;
        const uint8_t *b = row_block(p, slot[k], head, side);
        const int row = slot[k] & (p.c.page - 1);
        const uint8_t *c = b + r.off + row * 16 * r.w;
        if (side == 0) {
            word[k][0] = *reinterpret_cast<const uint32_t *>(c);
            word[k][1] = *reinterpret_cast<const uint32_t *>(c + 4 * r.w);
        } else {
            if (row & 2) c += r.turn;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                word[k][h] = *reinterpret_cast<const uint16_t *>(c + 4 * r.w * h) |
                             (uint32_t) * reinterpret_cast<const uint16_t *>(c + 4 * r.w * h + 2 * r.w) << 16;
        }
        s[k] = __half2float(*reinterpret_cast<const __half *>(b + code_bytes + (row * (p.c.dp / 32) + (r.el >> 5)) * 2));
    }
    const int64_t stride = side ? p.stride[1] : p.stride[0];
    uint8_t *dst = static_cast<uint8_t *>(side ? p.dst[1] : p.dst[0]) +
                   (r.token * stride + (int64_t)head * p.c.d + r.el) * type_bytes(TYPE);
    const uint64_t less = pair_f32(-8388616.0f, -8388616.0f);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        if (r.token + k * r.step >= p.n) break;
        const uint64_t s2 = pair_f32(s[k], s[k]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {  // 2^23 + code, less 2^23 + 8
                const float2 y = unpair_f32(mul_f32x2(
                    add_f32x2(pair_f32(__uint_as_float(((word[k][h] >> (4 * i)) & 15u) | 0x4B000000u),
                                       __uint_as_float(((word[k][h] >> (4 * i + 4)) & 15u) | 0x4B000000u)),
                              less),
                    s2));
                x[i] = y.x;
                x[i + 1] = y.y;
            }
            if (r.el + 8 * h < p.c.d) store8<TYPE>(dst + (k * r.step * stride + 8 * h) * type_bytes(TYPE), x);
        }
    }
}

static dim3 rows_grid(const Kv4View &c, int64_t n) {
    const int64_t tokens = (int64_t)(kRowsThreads / (c.dp / 16)) * kRows;  // a block
    return dim3((unsigned)((n + tokens - 1) / tokens), (unsigned)(2 * c.nkv));
}

int launch_kv4_append(const Kv4View &c, int type, const void *k, int64_t ks, const void *v, int64_t vs,
                      const int32_t *slots, int64_t n, cudaStream_t stream) {
    RowsK p = {c, {k, v}, {nullptr, nullptr}, {ks, vs}, slots, n, fault_word()};
    if (!p.fault) return QB_E_CUDA;
    auto *f = type == QB_T_F32 ? kv4_append_kernel<QB_T_F32>
              : type == QB_T_F16 ? kv4_append_kernel<QB_T_F16> : kv4_append_kernel<QB_T_BF16>;
    return launch_pdl(f, rows_grid(c, n), dim3(kRowsThreads), 0, stream, p);
}

int launch_kv4_read(const Kv4View &c, int type, const int32_t *slots, int64_t n, void *k, int64_t ks, void *v,
                    int64_t vs, cudaStream_t stream) {
    RowsK p = {c, {nullptr, nullptr}, {k, v}, {ks, vs}, slots, n, fault_word()};
    if (!p.fault) return QB_E_CUDA;
    auto *f = type == QB_T_F32 ? kv4_read_kernel<QB_T_F32>
              : type == QB_T_F16 ? kv4_read_kernel<QB_T_F16> : kv4_read_kernel<QB_T_BF16>;
    return launch_pdl(f, rows_grid(c, n), dim3(kRowsThreads), 0, stream, p);
}

}  // namespace qb
