// qb_kv_pages.cu -- the pages of a cache (qgemv.h: kv_pages_*): taking, sharing,
// giving back and moving them together, and the copies of their bytes.
//
// The state is a few thousand integers, so each call's decisions are made by
// one block of 1024 threads: what a request takes follows from prefix sums over
// the requests (or over a bitmap of the pages), never from the order in which
// threads arrive, so a state has one successor.  Fork and compact leave a
// list of (source, destination) pages in the workspace; a second launch copies
// them in every layer, bound by memory bandwidth.  A planning launch is latency: 7
// to 10 us for some hundreds to a thousand pages, chains of loads and block-wide sums.
// Compacting 32 layers after half of 32 sequences ended (258 MB moved): 102 us with
// the calls before it, of which 84 copy (6.2 TB/s read and written).
#include <algorithm>
#include <cstdint>

#include "qb_kv4.cuh"
#include "qb_kv_plan.cuh"

namespace qb {

// workspace: [0] pairs listed, [1] pages held (compact); then src, dst, map
struct PlanWs {
    int32_t *head, *src, *dst, *map;
};
static int64_t plan_pairs(int npages, int nrows) { return std::max(npages, nrows); }
int64_t kv_pages_ws(int npages, int nrows) {
    return (4 * (4 + 2 * plan_pairs(npages, nrows) + npages) + 15) / 16 * 16;
}
static PlanWs plan_ws(void *ws, int npages, int nrows) {
    PlanWs w;
    w.head = static_cast<int32_t *>(ws);
    w.src = w.head + 4;
    w.dst = w.src + plan_pairs(npages, nrows);
    w.map = w.dst + plan_pairs(npages, nrows);
    return w;
}

// ---------------------------------------------------------------- reset

__global__ void __launch_bounds__(256) kv_pages_reset_kernel(const PagesK p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t n = (int64_t)gridDim.x * blockDim.x, i0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    for (int64_t i = i0; i < p.npages; i += n) {
        p.free_pages[i] = (int32_t)(p.npages - 1 - i);
        p.refs[i] = 0;
    }
    for (int64_t i = i0; i < p.nrows; i += n) p.lens[i] = 0;
    for (int64_t i = i0; i < (int64_t)p.nrows * p.maxp; i += n) p.tables[i] = -1;
    if (i0 == 0) p.nfree[0] = p.npages;
}

// ---------------------------------------------------------------- extend

__global__ void __launch_bounds__(kPlanThreads) kv_pages_extend_kernel(const PagesK p, const int32_t *rows,
                                                                       const int32_t *counts, int n, int32_t *slots,
                                                                       int64_t nslots, int32_t *status) {
    __shared__ long long red[33];
    __shared__ int s_row[kPlanThreads], s_old[kPlanThreads], s_cnt[kPlanThreads], s_page[kPlanThreads];
    __shared__ long long s_tok[kPlanThreads];
    __shared__ int s_taken;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pshift = 31 - __clz(p.page);
    if (tid == 0) s_taken = 0;
    const int nfree = min(max(p.nfree[0], 0), p.npages);
    long long page_carry = 0, tok_carry = 0;
    __syncthreads();  // everyone has read nfree
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + tid;
        int row = -1, old = 0, cnt = 0, st = QB_OK;
        long long need = 0;
        if (i < n) {
            row = rows[i];
            cnt = counts[i];
            if (row < 0 || row >= p.nrows) {
                atomicOr(p.fault, kFaultIndex);
                row = -1;
                st = QB_E_ARG;
            } else {
                old = min(max(p.lens[row], 0), p.maxp * p.page);
            }
            if (cnt < 0) {
                cnt = 0;
                st = QB_E_ARG;
            }
            if (st == QB_OK && (long long)old + cnt > (long long)p.maxp * p.page) st = QB_E_PAGES;
            if (st == QB_OK) need = (((long long)old + cnt + p.page - 1) >> pshift) - ((old + p.page - 1) >> pshift);
        }
        long long pages, toks;
        const long long page0 = block_scan(need, red, pages) + page_carry;
        const long long tok0 = block_scan((long long)cnt, red, toks) + tok_carry;
        if (st == QB_OK && need > 0 && page0 + need > nfree) st = QB_E_PAGES;
        if (i < n) {
            status[i] = st;
            if (st == QB_OK) {
                p.lens[row] = old + cnt;
                if (need) atomicMax(&s_taken, (int)(page0 + need));
            }
        }
        s_row[tid] = st == QB_OK && i < n ? row : -1;
        s_old[tid] = old;
        s_cnt[tid] = cnt;
        s_page[tid] = (int)min(page0, (long long)p.npages);
        s_tok[tid] = tok0;
        page_carry += pages;
        tok_carry += toks;
        __syncthreads();
        // a warp a request: its pages, then its slots
        for (int r = warp; r < min(kPlanThreads, n - base); r += kPlanThreads / 32) {
            const int rr = s_row[r], o = s_old[r], c = s_cnt[r], pg0 = s_page[r];
            const long long t0 = s_tok[r];
            int32_t *tab = p.tables + (int64_t)max(rr, 0) * p.maxp;
            if (rr >= 0) {
                const int first = (o + p.page - 1) >> pshift, last = (int)(((long long)o + c + p.page - 1) >> pshift);
                for (int j = first + lane; j < last; j += 32) {
                    int pg = p.free_pages[nfree - 1 - (pg0 + j - first)];
                    if (pg < 0 || pg >= p.npages) {
                        atomicOr(p.fault, kFaultIndex);
                        pg = -1;
                    } else {
                        p.refs[pg] = 1;
                    }
                    tab[j] = pg;
                }
            }
            __syncwarp();
            // a refused request's count may be any: only the entries that `slots` has
            const int64_t room = kv_slots_room(c, t0, nslots);
            for (int64_t t = lane; t < room; t += 32) {
                int slot = -1;
                if (rr >= 0) {
                    const int pos = o + (int)t, pg = tab[pos >> pshift];
                    if (pg >= 0) slot = (pg << pshift) + (pos & (p.page - 1));
                }
                slots[t0 + t] = slot;
            }
            if (lane == 0 && room < c) atomicOr(p.fault, kFaultIndex);
        }
        __syncthreads();
    }
    if (tid == 0) p.nfree[0] = nfree - s_taken;
}

// ---------------------------------------------------------------- fork

__global__ void __launch_bounds__(kPlanThreads) kv_pages_fork_kernel(const PagesK p, const int32_t *parents,
                                                                     const int32_t *children, int n, int32_t *status,
                                                                     const PlanWs w) {
    __shared__ int red[33];
    __shared__ int s_par[kPlanThreads], s_chi[kPlanThreads], s_page[kPlanThreads], s_len[kPlanThreads];
    __shared__ int s_taken;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pshift = 31 - __clz(p.page);
    if (tid == 0) s_taken = 0;
    const int nfree = min(max(p.nfree[0], 0), p.npages);
    int carry = 0;
    __syncthreads();
    for (int base = 0; base < n; base += kPlanThreads) {
        const int i = base + tid;
        int par = -1, chi = -1, len = 0, st = QB_OK;
        if (i < n) {
            par = parents[i];
            chi = children[i];
            if (par < 0 || par >= p.nrows || chi < 0 || chi >= p.nrows) {
                atomicOr(p.fault, kFaultIndex);
                st = QB_E_ARG;
            } else {
                len = min(max(p.lens[par], 0), p.maxp * p.page);
                if (p.lens[chi] != 0) st = QB_E_ARG;
            }
        }
        const int need = i < n && st == QB_OK && (len & (p.page - 1)) != 0;
        int total;
        const int rank = block_scan(need, red, total) + carry;
        carry += total;
        int pg = -1;
        if (need) {
            if (rank < nfree) {
                pg = p.free_pages[nfree - 1 - rank];
                const int old = p.tables[(int64_t)par * p.maxp + (len >> pshift)];
                const bool bad = pg < 0 || pg >= p.npages || old < 0 || old >= p.npages;
                if (bad) atomicOr(p.fault, kFaultIndex);
                w.src[rank] = bad ? -1 : old;
                w.dst[rank] = bad ? -1 : pg;
                if (!bad) p.refs[pg] = 1;
                if (bad) pg = -1;
                atomicMax(&s_taken, rank + 1);
            } else {
                st = QB_E_PAGES;
            }
        }
        if (i < n) status[i] = st;
        s_par[tid] = i < n && st == QB_OK ? par : -1;
        s_chi[tid] = chi;
        s_page[tid] = pg;
        s_len[tid] = len;
        __syncthreads();  // also: every child's length has been looked at
        for (int r = warp; r < min(kPlanThreads, n - base); r += kPlanThreads / 32) {
            if (s_par[r] < 0) continue;
            const int l = s_len[r], full = l >> pshift;
            const int32_t *from = p.tables + (int64_t)s_par[r] * p.maxp;
            int32_t *to = p.tables + (int64_t)s_chi[r] * p.maxp;
            for (int j = lane; j < p.maxp; j += 32) {
                int v = -1;
                if (j < full) {
                    v = from[j];
                    if (v >= 0 && v < p.npages)
                        atomicAdd(p.refs + v, 1);
                    else
                        atomicOr(p.fault, kFaultIndex);
                } else if (j == full && (l & (p.page - 1))) {
                    v = s_page[r];
                }
                to[j] = v;
            }
            if (lane == 0) p.lens[s_chi[r]] = l;
        }
        __syncthreads();
    }
    if (tid == 0) {
        p.nfree[0] = nfree - s_taken;
        w.head[0] = s_taken;
    }
}

// ---------------------------------------------------------------- free

__global__ void __launch_bounds__(kPlanThreads) kv_pages_free_kernel(const PagesK p, const int32_t *rows, int n) {
    extern __shared__ uint32_t freed[];  // a bit a page
    __shared__ int red[33];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int words = (p.npages + 31) / 32, pshift = 31 - __clz(p.page);
    for (int i = tid; i < words; i += kPlanThreads) freed[i] = 0;
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();
    const int nfree = min(max(p.nfree[0], 0), p.npages);
    for (int r = warp; r < n; r += kPlanThreads / 32) {
        const int row = rows[r];
        if (row < 0 || row >= p.nrows) {
            if (lane == 0) atomicOr(p.fault, kFaultIndex);
            continue;
        }
        int32_t *tab = p.tables + (int64_t)row * p.maxp;
        const int held = min((int)(((long long)max(p.lens[row], 0) + p.page - 1) >> pshift), p.maxp);
        for (int j = lane; j < p.maxp; j += 32) {
            if (j < held) {
                const int pg = tab[j];
                if (pg < 0 || pg >= p.npages)
                    atomicOr(p.fault, kFaultIndex);
                else if (atomicSub(p.refs + pg, 1) == 1)
                    atomicOr(freed + (pg >> 5), 1u << (pg & 31));
            }
            tab[j] = -1;
        }
        __syncwarp();  // every lane has read the length
        if (lane == 0) p.lens[row] = 0;
    }
    __syncthreads();
    give_back(p, freed, words, nfree, red);
}

// ---------------------------------------------------------------- compact

__global__ void __launch_bounds__(kPlanThreads) kv_pages_compact_kernel(const PagesK p, const PlanWs w) {
    extern __shared__ uint32_t held[];  // a bit a page
    __shared__ int red[33];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int words = (p.npages + 31) / 32;
    for (int i = tid; i < words * 32; i += kPlanThreads) {
        const uint32_t b = __ballot_sync(0xFFFFFFFFu, i < p.npages && p.refs[i] > 0);
        if (lane == 0) held[i >> 5] = b;
    }
    __syncthreads();
    const int per = (words + kPlanThreads - 1) / kPlanThreads, w0 = min(tid * per, words), w1 = min(w0 + per, words);
    int cnt = 0;
    for (int i = w0; i < w1; ++i) cnt += __popc(held[i]);
    int used;
    block_scan(cnt, red, used);
    // pages below `used` of a word: all, none or the low ones
    auto below = [&](int i) -> uint32_t {
        const int k = used - i * 32;
        return k >= 32 ? 0xFFFFFFFFu : k <= 0 ? 0u : (1u << k) - 1u;
    };
    int moves = 0, holes = 0;
    for (int i = w0; i < w1; ++i) {
        moves += __popc(held[i] & ~below(i));
        holes += __popc(~held[i] & below(i));
    }
    int nmoves, nholes;
    int m = block_scan(moves, red, nmoves), h = block_scan(holes, red, nholes);
    for (int i = w0; i < w1; ++i) {
        for (uint32_t b = held[i] & ~below(i); b; b &= b - 1) w.src[m++] = i * 32 + __ffs(b) - 1;
        for (uint32_t b = ~held[i] & below(i); b; b &= b - 1) w.dst[h++] = i * 32 + __ffs(b) - 1;
    }
    __syncthreads();
    for (int i = tid; i < nmoves; i += kPlanThreads) {
        const int from = w.src[i], to = w.dst[i];
        w.map[from] = to;
        p.refs[to] = p.refs[from];
        p.refs[from] = 0;
    }
    for (int i = tid; i < p.npages - used; i += kPlanThreads) p.free_pages[i] = p.npages - 1 - i;
    if (tid == 0) {
        p.nfree[0] = p.npages - used;
        w.head[0] = nmoves;
        w.head[1] = used;
    }
}

// ---------------------------------------------------------------- copies

struct CopyK {
    uint8_t *data;
    int nlayers;
    int64_t npages, page_bytes;
    const int32_t *src, *dst;
    const int32_t *count;  // NULL: n
    int n;
    int *fault;
    // compact: table entries from head[1] up are looked up in map
    int32_t *tables;
    int64_t entries;
    const int32_t *map;
};

constexpr int kCopyThreads = 256, kCopyVecs = 4;  // 16 KB a block and turn

__global__ void __launch_bounds__(kCopyThreads) kv_pages_copy_kernel(const CopyK p) {
    // no early launch_dependents: the pages may be those of the int8 cache, whose
    // score kernel reads key rows before its own pdl_wait
    pdl_wait();
    const int n = p.count ? p.count[0] : p.n;
    const int64_t vecs = p.page_bytes / 16;
    constexpr int kTurn = kCopyThreads * kCopyVecs;
    const int64_t turns = (vecs + kTurn - 1) / kTurn;
    const int64_t total = (int64_t)n * p.nlayers * turns;
    for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
        const int64_t page_i = i / turns, turn = i - page_i * turns;
        const int layer = (int)(page_i / n), pair = (int)(page_i - (int64_t)layer * n);
        const int s = p.src[pair], d = p.dst[pair];
        if (s < 0 || d < 0 || s >= p.npages || d >= p.npages) {
            if (threadIdx.x == 0) atomicOr(p.fault, kFaultIndex);
            continue;
        }
        const int64_t layer_off = (int64_t)layer * p.npages;
        const uint4 *from = reinterpret_cast<const uint4 *>(p.data + (layer_off + s) * p.page_bytes);
        uint4 *to = reinterpret_cast<uint4 *>(p.data + (layer_off + d) * p.page_bytes);
        uint4 v[kCopyVecs];
        const int64_t at = turn * kTurn + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k)
            if (at + k * kCopyThreads < vecs) v[k] = __ldcs(from + at + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < kCopyVecs; ++k)
            if (at + k * kCopyThreads < vecs) __stcs(to + at + k * kCopyThreads, v[k]);
    }
    if (p.map) {
        const int used = p.count[1];
        for (int64_t i = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; i < p.entries;
             i += (int64_t)gridDim.x * kCopyThreads) {
            const int v = p.tables[i];
            if (v < used) continue;
            if (v < p.npages)
                p.tables[i] = p.map[v];
            else
                atomicOr(p.fault, kFaultIndex);
        }
    }
}

// ---------------------------------------------------------------- launchers

int launch_kv_pages_reset(const qb_kv_pages &p, cudaStream_t stream) {
    const PagesK k = pages_k(p);
    const int64_t n = std::max<int64_t>(p.npages, (int64_t)p.nrows * p.maxp);
    return launch_pdl(kv_pages_reset_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 4096)), dim3(256), 0,
                      stream, k);
}

int launch_kv_pages_extend(const qb_kv_pages &p, const int32_t *rows, const int32_t *counts, int n, int32_t *slots,
                           int64_t nslots, int32_t *status, cudaStream_t stream) {
    const PagesK k = pages_k(p);
    if (!k.fault) return QB_E_CUDA;
    return launch_pdl(kv_pages_extend_kernel, dim3(1), dim3(kPlanThreads), 0, stream, k, rows, counts, n, slots,
                      nslots, status);
}

static int launch_copy(const CopyK &c, int64_t most_pages, cudaStream_t stream) {
    const int64_t turns = (c.page_bytes / 16 + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs);
    const int64_t blocks = std::min<int64_t>(most_pages * c.nlayers * turns, (int64_t)num_sms() * 8);
    return launch_pdl(kv_pages_copy_kernel, dim3((unsigned)std::max<int64_t>(blocks, 1)), dim3(kCopyThreads), 0,
                      stream, c);
}

int launch_kv_pages_fork(const qb_kv_pages &p, void *data, int nlayers, int64_t page_bytes, const int32_t *parents,
                         const int32_t *children, int n, int32_t *status, void *ws, cudaStream_t stream) {
    const PagesK k = pages_k(p);
    if (!k.fault) return QB_E_CUDA;
    const PlanWs w = plan_ws(ws, p.npages, p.nrows);
    const int rc = launch_pdl(kv_pages_fork_kernel, dim3(1), dim3(kPlanThreads), 0, stream, k, parents, children, n,
                              status, w);
    if (rc) return rc;
    CopyK c = {};
    c.data = static_cast<uint8_t *>(data);
    c.nlayers = nlayers;
    c.npages = p.npages;
    c.page_bytes = page_bytes;
    c.src = w.src;
    c.dst = w.dst;
    c.count = w.head;
    c.fault = k.fault;
    return launch_copy(c, n, stream);
}

int launch_kv_pages_free(const qb_kv_pages &p, const int32_t *rows, int n, cudaStream_t stream) {
    const PagesK k = pages_k(p);
    if (!k.fault) return QB_E_CUDA;
    const int smem = (p.npages + 31) / 32 * 4;
    if (ensure_smem_limit(reinterpret_cast<const void *>(kv_pages_free_kernel), smem) != QB_OK) return QB_E_CUDA;
    return launch_pdl(kv_pages_free_kernel, dim3(1), dim3(kPlanThreads), (size_t)smem, stream, k, rows, n);
}

int launch_kv_pages_compact(const qb_kv_pages &p, void *data, int nlayers, int64_t page_bytes, void *ws,
                            cudaStream_t stream) {
    const PagesK k = pages_k(p);
    if (!k.fault) return QB_E_CUDA;
    const PlanWs w = plan_ws(ws, p.npages, p.nrows);
    const int smem = (p.npages + 31) / 32 * 4;
    if (ensure_smem_limit(reinterpret_cast<const void *>(kv_pages_compact_kernel), smem) != QB_OK) return QB_E_CUDA;
    const int rc = launch_pdl(kv_pages_compact_kernel, dim3(1), dim3(kPlanThreads), (size_t)smem, stream, k, w);
    if (rc) return rc;
    CopyK c = {};
    c.data = static_cast<uint8_t *>(data);
    c.nlayers = nlayers;
    c.npages = p.npages;
    c.page_bytes = page_bytes;
    c.src = w.src;
    c.dst = w.dst;
    c.count = w.head;
    c.fault = k.fault;
    c.tables = p.tables;
    c.entries = (int64_t)p.nrows * p.maxp;
    c.map = w.map;
    return launch_copy(c, (p.npages + 1) / 2, stream);
}

int launch_kv_pages_copy(void *data, int nlayers, int64_t npages, int64_t page_bytes, const int32_t *src,
                         const int32_t *dst, int n, cudaStream_t stream) {
    CopyK c = {};
    c.data = static_cast<uint8_t *>(data);
    c.nlayers = nlayers;
    c.npages = npages;
    c.page_bytes = page_bytes;
    c.src = src;
    c.dst = dst;
    c.n = n;
    c.fault = fault_word();
    if (!c.fault) return QB_E_CUDA;
    return launch_copy(c, n, stream);
}

}  // namespace qb
