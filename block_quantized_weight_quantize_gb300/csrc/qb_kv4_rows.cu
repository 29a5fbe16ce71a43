// qb_kv4_rows.cu -- rows into and out of the paged 4-bit cache (qgemv.h:
// kv4_append, kv4_read).
//
// A thread takes 8 consecutive elements of one row: one word of a key row, two
// halves of a value row; four neighbouring threads hold a group of 32 and find
// its step by two shuffles.  Bound by memory: each element is read once and
// its half byte written once (or the reverse).
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

// The thread's place: row (token and key head) and 8-element piece of it.
struct RowPlace {
    int64_t token;
    int head, oct;
    bool live;
};
__device__ __forceinline__ RowPlace row_place(const RowsK &p) {
    const int octs = p.c.dp / 8;  // 8, 16 or 32: a power of two
    const int sh = octs == 8 ? 3 : octs == 16 ? 4 : 5;
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    RowPlace r;
    r.oct = (int)(i & (octs - 1));
    const int64_t row = i >> sh;
    r.token = row / p.c.nkv;
    r.head = (int)(row - r.token * p.c.nkv);
    r.live = r.token < p.n;
    return r;
}

template <int TYPE>
__global__ void __launch_bounds__(256) kv4_append_kernel(const RowsK p) {
    pdl_launch_dependents();
    pdl_wait();
    const RowPlace r = row_place(p);
    const int side = blockIdx.y, page = p.c.page, w = min(p.c.dp / 32, 4);
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    int slot = -1;
    if (r.live) {
        slot = p.slots[r.token];
        if ((slot >> p.c.pshift) >= p.c.npages) {
            atomicOr(p.fault, kFaultIndex);
            slot = -1;
        }
        if (r.oct * 8 < p.c.d)
            load8<TYPE>(static_cast<const uint8_t *>(p.src[side]) +
                            (r.token * p.stride[side] + (int64_t)r.head * p.c.d + r.oct * 8) * type_bytes(TYPE),
                        x);
    }
    // the group's extremes: fmaxf and fminf pass NaN over
    float hi = 0.0f, lo = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        hi = fmaxf(hi, x[i]);
        lo = fminf(lo, x[i]);
    }
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    }
    const __half step = __float2half_rn((hi >= -lo ? hi : lo) * -0.125f);
    const float s = __half2float(step);
    const float inv = s == 0.0f ? 0.0f : __frcp_rn(s);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float y = fminf(fmaxf(rintf(__fmul_rn(x[i], inv)), -8.0f), 7.0f);
        const int c = x[i] * inv == x[i] * inv ? (int)y : 0;  // a NaN product: zero
        word |= (uint32_t)(c + 8) << (4 * i);
    }
    if (slot < 0) return;
    const int pg = slot >> p.c.pshift, row = slot & (page - 1);
    uint8_t *b = p.c.data + ((int64_t)pg * p.c.nkv + r.head) * p.c.block_bytes;
    const int code_bytes = page * p.c.dp / 2, step_bytes = page * p.c.dp / 16;
    if (side) b += code_bytes + step_bytes;
    if (side == 0) {
        *reinterpret_cast<uint32_t *>(b + kv4_key_word(page, w, row, r.oct)) = word;
    } else {
        *reinterpret_cast<uint16_t *>(b + kv4_value_half(page, w, row, r.oct, 0)) = (uint16_t)word;
        *reinterpret_cast<uint16_t *>(b + kv4_value_half(page, w, row, r.oct, 1)) = (uint16_t)(word >> 16);
    }
    if ((r.oct & 3) == 0)
        *reinterpret_cast<__half *>(b + code_bytes + (row * (p.c.dp / 32) + (r.oct >> 2)) * 2) = step;
}

template <int TYPE>
__global__ void __launch_bounds__(256) kv4_read_kernel(const RowsK p) {
    pdl_launch_dependents();
    pdl_wait();
    const RowPlace r = row_place(p);
    const int side = blockIdx.y, page = p.c.page, w = min(p.c.dp / 32, 4);
    if (!r.live || r.oct * 8 >= p.c.d) return;
    int slot = p.slots[r.token];
    if ((slot >> p.c.pshift) >= p.c.npages) {
        atomicOr(p.fault, kFaultIndex);
        slot = -1;
    }
    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (slot >= 0) {
        const int pg = slot >> p.c.pshift, row = slot & (page - 1);
        const uint8_t *b = p.c.data + ((int64_t)pg * p.c.nkv + r.head) * p.c.block_bytes;
        const int code_bytes = page * p.c.dp / 2, step_bytes = page * p.c.dp / 16;
        if (side) b += code_bytes + step_bytes;
        uint32_t word;
        if (side == 0) {
            word = *reinterpret_cast<const uint32_t *>(b + kv4_key_word(page, w, row, r.oct));
        } else {
            word = *reinterpret_cast<const uint16_t *>(b + kv4_value_half(page, w, row, r.oct, 0)) |
                   (uint32_t) * reinterpret_cast<const uint16_t *>(b + kv4_value_half(page, w, row, r.oct, 1)) << 16;
        }
        const float s = __half2float(
            *reinterpret_cast<const __half *>(b + code_bytes + (row * (p.c.dp / 32) + (r.oct >> 2)) * 2));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)((int)((word >> (4 * i)) & 15u) - 8) * s;
    }
    store8<TYPE>(static_cast<uint8_t *>(p.dst[side]) +
                     (r.token * p.stride[side] + (int64_t)r.head * p.c.d + r.oct * 8) * type_bytes(TYPE),
                 x);
}

static dim3 rows_grid(const Kv4View &c, int64_t n) {
    return dim3((unsigned)((n * c.nkv * (c.dp / 8) + 255) / 256), 2);
}

int launch_kv4_append(const Kv4View &c, int type, const void *k, int64_t ks, const void *v, int64_t vs,
                      const int32_t *slots, int64_t n, cudaStream_t stream) {
    RowsK p = {c, {k, v}, {nullptr, nullptr}, {ks, vs}, slots, n, fault_word()};
    if (!p.fault) return QB_E_CUDA;
    auto *f = type == QB_T_F32 ? kv4_append_kernel<QB_T_F32>
              : type == QB_T_F16 ? kv4_append_kernel<QB_T_F16> : kv4_append_kernel<QB_T_BF16>;
    return launch_pdl(f, rows_grid(c, n), dim3(256), 0, stream, p);
}

int launch_kv4_read(const Kv4View &c, int type, const int32_t *slots, int64_t n, void *k, int64_t ks, void *v,
                    int64_t vs, cudaStream_t stream) {
    RowsK p = {c, {nullptr, nullptr}, {k, v}, {ks, vs}, slots, n, fault_word()};
    if (!p.fault) return QB_E_CUDA;
    auto *f = type == QB_T_F32 ? kv4_read_kernel<QB_T_F32>
              : type == QB_T_F16 ? kv4_read_kernel<QB_T_F16> : kv4_read_kernel<QB_T_BF16>;
    return launch_pdl(f, rows_grid(c, n), dim3(256), 0, stream, p);
}

}  // namespace qb
