// qb_kv4_api.cu -- the C entry points of the paged 4-bit cache (qgemv.h):
// argument checks on the host, then the launches on the caller's stream.
#include <cmath>
#include <cstdint>

#include "qb_kv4.cuh"

using namespace qb;

namespace {

bool off(const void *p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

bool page_ok(int page) { return page == 16 || page == 32 || page == 64; }

int check_cache(const qb_kv4 *c) {
    if (!c || !c->data || off(c->data, 16) || !page_ok(c->page) || c->npages < 1 || c->nkv < 1 || c->nkv > 1024 ||
        c->d < 8 || c->d > 256 || c->d % 8 != 0 || (int64_t)c->npages * c->page >= (int64_t(1) << 31))
        return QB_E_ARG;
    return QB_OK;
}

// n token rows of `width` elements with `stride` elements between them
bool rows_bad(const void *p, int64_t stride, int64_t width, int es) {
    return !p || off(p, 16) || stride < width || stride > (int64_t(1) << 40) || stride * es % 16 != 0;
}

bool type_ok(qb_type t) { return t == QB_T_F32 || t == QB_T_F16 || t == QB_T_BF16; }

int check_rows(const qb_kv4 *c, qb_type type, const void *k, int64_t ks, const void *v, int64_t vs,
               const int32_t *slots, int64_t n) {
    if (check_cache(c) || !type_ok(type) || n < 0 || n >= (int64_t(1) << 31)) return QB_E_ARG;
    if (n == 0) return QB_OK;  // empty arrays may have no address
    if (!slots || off(slots, 4)) return QB_E_ARG;
    const int64_t width = (int64_t)c->nkv * c->d;
    const int es = type_bytes(type);
    if (rows_bad(k, ks, width, es) || rows_bad(v, vs, width, es)) return QB_E_ARG;
    return QB_OK;
}

int check_pages(const qb_kv_pages *p) {
    if (!p || !p->nfree || !p->free_pages || !p->refs || !p->lens || !p->tables) return QB_E_ARG;
    if (off(p->nfree, 4) || off(p->free_pages, 4) || off(p->refs, 4) || off(p->lens, 4) || off(p->tables, 4))
        return QB_E_ARG;
    if (!page_ok(p->page) || p->npages < 1 || p->npages > (1 << 20) || p->nrows < 1 || p->nrows > (1 << 20) ||
        p->maxp < 1 || (int64_t)p->maxp * p->page >= (int64_t(1) << 31))
        return QB_E_ARG;
    return QB_OK;
}

bool data_bad(const void *data, int nlayers, int64_t page_bytes) {
    return !data || off(data, 16) || nlayers < 1 || nlayers > 65535 || page_bytes < 16 || page_bytes % 16 != 0 ||
           page_bytes > (int64_t(1) << 31);
}

}  // namespace

extern "C" {

int64_t kv4_block_bytes(int page, int d) {
    if (!page_ok(page) || d < 8 || d > 256 || d % 8 != 0) return QB_E_ARG;
    return kv4_block(page, kv4_padded(d));
}

int kv4_append(const qb_kv4 *cache, qb_type type, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
               const int32_t *slots, int64_t n, void *stream) {
    if (const int rc = check_rows(cache, type, k, k_stride, v, v_stride, slots, n)) return rc;
    if (n == 0) return QB_OK;
    return launch_kv4_append(kv4_view(*cache), type, k, k_stride, v, v_stride, slots, n,
                             static_cast<cudaStream_t>(stream));
}

int kv4_read(const qb_kv4 *cache, qb_type type, const int32_t *slots, int64_t n, void *k, int64_t k_stride, void *v,
             int64_t v_stride, void *stream) {
    if (const int rc = check_rows(cache, type, k, k_stride, v, v_stride, slots, n)) return rc;
    if (n == 0) return QB_OK;
    return launch_kv4_read(kv4_view(*cache), type, slots, n, k, k_stride, v, v_stride,
                           static_cast<cudaStream_t>(stream));
}

int64_t kv4_attn_workspace_bytes(const qb_kv4 *cache, int nh) {
    if (!cache || cache->nkv < 1 || cache->nkv > 1024 || cache->d < 8 || cache->d > 256 || cache->d % 8 != 0 ||
        nh < 1 || nh > 4096 || nh % cache->nkv != 0)
        return QB_E_ARG;
    return kv4_attn_ws(kv4_padded(cache->d));
}

int kv4_attn(const qb_kv4 *cache, const qb_kv_seqs *seqs, qb_type type, const void *q, int64_t q_stride,
             int64_t ntok, int nh, float scale, int window, void *out, int64_t out_stride, float *lse,
             void *workspace, size_t workspace_bytes, void *stream) {
    if (check_cache(cache) || !seqs || !type_ok(type) || window < 0 || !std::isfinite(scale)) return QB_E_ARG;
    if (!seqs->tables || !seqs->lens || off(seqs->tables, 4) || off(seqs->lens, 4) || off(seqs->rows, 4) ||
        off(seqs->q_start, 4))
        return QB_E_ARG;
    if (seqs->nseq < 0 || seqs->nseq > 8192 || (seqs->nseq == 0 && ntok != 0) || seqs->nrows < 1 || seqs->maxp < 1 ||
        (int64_t)seqs->maxp * cache->page >= (int64_t(1) << 31))
        return QB_E_ARG;
    if (!seqs->rows && seqs->nseq > seqs->nrows) return QB_E_ARG;
    if (nh < 1 || nh > 4096 || nh % cache->nkv != 0 || ntok < 0 || ntok > (int64_t(1) << 24) ||
        ntok * nh > (int64_t(1) << 30))
        return QB_E_ARG;
    if (!seqs->q_start && ntok != seqs->nseq) return QB_E_ARG;
    if (ntok == 0) return QB_OK;
    const int64_t width = (int64_t)nh * cache->d;
    const int es = type_bytes(type);
    if (rows_bad(q, q_stride, width, es) || rows_bad(out, out_stride, width, es) || off(lse, 4)) return QB_E_ARG;
    const int64_t need = kv4_attn_workspace_bytes(cache, nh);
    if (need < 0) return (int)need;
    if (!workspace || off(workspace, 16) || (int64_t)workspace_bytes < need) return QB_E_ARG;
    Kv4AttnArgs a = {};
    a.c = kv4_view(*cache);
    a.s = *seqs;
    a.type = type;
    a.q = q;
    a.q_stride = q_stride;
    a.ntok = ntok;
    a.nh = nh;
    a.scale = scale;
    a.window = window;
    a.out = out;
    a.out_stride = out_stride;
    a.lse = lse;
    a.ws = static_cast<uint8_t *>(workspace);
    a.fault = fault_word();
    if (!a.fault) return QB_E_CUDA;
    return launch_kv4_attn(a, static_cast<cudaStream_t>(stream));
}

int64_t kv_pages_workspace_bytes(const qb_kv_pages *pages) {
    if (const int rc = check_pages(pages)) return rc;
    return kv_pages_ws(pages->npages, pages->nrows);
}

int kv_pages_reset(const qb_kv_pages *pages, void *stream) {
    if (const int rc = check_pages(pages)) return rc;
    return launch_kv_pages_reset(*pages, static_cast<cudaStream_t>(stream));
}

int kv_pages_extend(const qb_kv_pages *pages, const int32_t *rows, const int32_t *counts, int n, int32_t *slots,
                    int64_t nslots, int32_t *status, void *stream) {
    if (const int rc = check_pages(pages)) return rc;
    if (n < 0 || n > pages->nrows || nslots < 0) return QB_E_ARG;
    if (n == 0) return QB_OK;
    if (!rows || !counts || (!slots && nslots > 0) || !status || off(rows, 4) || off(counts, 4) || off(slots, 4) ||
        off(status, 4))
        return QB_E_ARG;
    return launch_kv_pages_extend(*pages, rows, counts, n, slots, nslots, status, static_cast<cudaStream_t>(stream));
}

int kv_pages_fork(const qb_kv_pages *pages, void *data, int nlayers, int64_t page_bytes, const int32_t *parents,
                  const int32_t *children, int n, int32_t *status, void *workspace, size_t workspace_bytes,
                  void *stream) {
    if (const int rc = check_pages(pages)) return rc;
    if (data_bad(data, nlayers, page_bytes) || n < 0 || n > pages->nrows) return QB_E_ARG;
    if (n == 0) return QB_OK;
    if (!parents || !children || !status || off(parents, 4) || off(children, 4) || off(status, 4)) return QB_E_ARG;
    if (!workspace || off(workspace, 16) || (int64_t)workspace_bytes < kv_pages_ws(pages->npages, pages->nrows))
        return QB_E_ARG;
    return launch_kv_pages_fork(*pages, data, nlayers, page_bytes, parents, children, n, status, workspace,
                                static_cast<cudaStream_t>(stream));
}

int kv_pages_free(const qb_kv_pages *pages, const int32_t *rows, int n, void *stream) {
    if (const int rc = check_pages(pages)) return rc;
    if (n < 0 || n > pages->nrows) return QB_E_ARG;
    if (n == 0) return QB_OK;
    if (!rows || off(rows, 4)) return QB_E_ARG;
    return launch_kv_pages_free(*pages, rows, n, static_cast<cudaStream_t>(stream));
}

int kv_pages_compact(const qb_kv_pages *pages, void *data, int nlayers, int64_t page_bytes, void *workspace,
                     size_t workspace_bytes, void *stream) {
    if (const int rc = check_pages(pages)) return rc;
    if (data_bad(data, nlayers, page_bytes)) return QB_E_ARG;
    if (!workspace || off(workspace, 16) || (int64_t)workspace_bytes < kv_pages_ws(pages->npages, pages->nrows))
        return QB_E_ARG;
    return launch_kv_pages_compact(*pages, data, nlayers, page_bytes, workspace, static_cast<cudaStream_t>(stream));
}

int kv_pages_copy(void *data, int nlayers, int64_t npages, int64_t page_bytes, const int32_t *src, const int32_t *dst,
                  int n, void *stream) {
    if (data_bad(data, nlayers, page_bytes) || npages < 1 || npages > (1 << 20) || n < 0 || n > npages) return QB_E_ARG;
    if (n == 0) return QB_OK;
    if (!src || !dst || off(src, 4) || off(dst, 4)) return QB_E_ARG;
    return launch_kv_pages_copy(data, nlayers, npages, page_bytes, src, dst, n, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
