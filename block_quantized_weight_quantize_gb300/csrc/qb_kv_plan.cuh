// qb_kv_plan.cuh -- what the kernels that change the pages' state share (qb_kv_pages.cu, qb_kv4_keep.cu).
#pragma once

#include <cstdint>

#include "qb_kv4.cuh"

namespace qb {

constexpr int kPlanThreads = 1024;

struct PagesK {
    int32_t *nfree, *free_pages, *refs, *lens, *tables;
    int page, npages, nrows, maxp;
    int *fault;
};

inline PagesK pages_k(const qb_kv_pages &p) {
    return PagesK{p.nfree, p.free_pages, p.refs, p.lens, p.tables, p.page, p.npages, p.nrows, p.maxp, fault_word()};
}

// Exclusive prefix sum of x over the block's threads, and the total; red has 33 entries.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *red, T &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();  // red of an earlier scan has been read
    if (lane == 31) red[warp] = s;
    __syncthreads();
    if (warp == 0) {
        T y = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T z = __shfl_up_sync(0xFFFFFFFFu, y, o);
            if (lane >= o) y += z;
        }
        red[lane] = y;
    }
    __syncthreads();
    total = red[31];
    return s - x + (warp ? red[warp - 1] : T(0));
}

// The pages whose bits are set go back to the stack in ascending order, behind its `nfree` entries; by a whole block.
__device__ __forceinline__ void give_back(const PagesK &p, const uint32_t *freed, int words, int nfree, int *red) {
    const int tid = threadIdx.x;
    const int per = (words + kPlanThreads - 1) / kPlanThreads, w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int cnt = 0;
    for (int i = w0; i < w1; ++i) cnt += __popc(freed[i]);
    int total;
    int at = nfree + block_scan(cnt, red, total);
    for (int i = w0; i < w1; ++i)
        for (uint32_t b = freed[i]; b; b &= b - 1) {
            if (at < p.npages) p.free_pages[at] = i * 32 + __ffs(b) - 1;
            ++at;
        }
    if (tid == 0) p.nfree[0] = min(nfree + total, p.npages);
}

}  // namespace qb
