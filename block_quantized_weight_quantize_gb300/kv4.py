"""Binding of the paged 4-bit key/value cache: rows in and out, attention over
it, and its pages (``kv4_*`` and ``kv_pages_*`` of ``include/qgemv.h``).

A cache, its sequences and its pages are small handles made once; each call
marshals pointers and raises on a non-zero status.  Tensors keep the layouts
of the header: caches uint8 [npages, nkv * kv4_block_bytes(page, d)], rows
[n, nkv, d] and queries [ntok, nh, d] of float32, float16 or bfloat16 (the last
two axes contiguous), int32 for everything that counts pages or tokens.  The
tensors of a call lie on one device, the current one, where the library launches.
"""
from __future__ import annotations

import ctypes

import torch

from . import _check, lib, QbError

T_F32, T_F16, T_BF16 = 0, 1, 2  # QB_T_*
_TYPE = {torch.float32: T_F32, torch.float16: T_F16, torch.bfloat16: T_BF16}


class _CKv4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("npages", ctypes.c_int), ("page", ctypes.c_int), ("nkv", ctypes.c_int),
                ("d", ctypes.c_int)]


class _CSeqs(ctypes.Structure):
    _fields_ = [("tables", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("rows", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p), ("nrows", ctypes.c_int), ("maxp", ctypes.c_int), ("nseq", ctypes.c_int)]


class _CPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("nfree", "free_pages", "refs", "lens", "tables")] + \
               [(n, ctypes.c_int) for n in ("page", "npages", "nrows", "maxp")]


_P, _I, _L = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
_SIGNATURES = {
    "kv4_block_bytes": ([_I, _I], _L),
    "kv4_append": ([_P, _I, _P, _L, _P, _L, _P, _L, _P], _I),
    "kv4_read": ([_P, _I, _P, _L, _P, _L, _P, _L, _P], _I),
    "kv4_attn_workspace_bytes": ([_P, _I], _L),
    "kv4_attn": ([_P, _P, _I, _P, _L, _L, _I, ctypes.c_float, _I, _P, _L, _P, _P, ctypes.c_size_t, _P], _I),
    "kv_pages_workspace_bytes": ([_P], _L),
    "kv_pages_reset": ([_P, _P], _I),
    "kv_pages_extend": ([_P, _P, _P, _I, _P, _L, _P, _P], _I),
    "kv_pages_fork": ([_P, _P, _I, _L, _P, _P, _I, _P, _P, ctypes.c_size_t, _P], _I),
    "kv_pages_free": ([_P, _P, _I, _P], _I),
    "kv_pages_compact": ([_P, _P, _I, _L, _P, ctypes.c_size_t, _P], _I),
    "kv_pages_copy": ([_P, _I, _L, _L, _P, _P, _I, _P], _I),
}

class _Calls:
    """The library's entry points with their signatures set, looked up once."""

    def __getattr__(self, name):
        f = getattr(lib(), name)
        f.argtypes, f.restype = _SIGNATURES[name]
        setattr(self, name, f)
        return f


_c = _Calls()
_raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _stream(stream, dev: int) -> int:
    """Handle of `stream`, or of the current one, for a call whose tensors lie on device `dev`."""
    if dev != _current_device():
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{_current_device()}")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _workspace(nbytes: int, like, stream):
    """A workspace for one call on `stream` (None: the current one) of the device of `like`.  It is that stream's memory from the
    start: a block that the current stream has given back may still be in use by what is queued there, and one of this
    stream's is given out again only to calls that follow on it."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _bytes(n: int, where: str) -> int:
    if n < 0:
        raise QbError(int(n), where)
    return int(n)


def _on(t, what: str, dev=None) -> int:
    """The device that t lies on: `dev`, where that is given."""
    d = t.get_device()
    if d != dev:
        if d < 0:
            raise ValueError(f"{what}: device memory expected, got a CPU tensor")
        if dev is not None:
            raise ValueError(f"{what}: on cuda:{d}, where the call's other tensors are on cuda:{dev}")
    return d


def _dev(t, dtype, what: str, dev: int):
    """Address of a contiguous tensor of `dtype` on device `dev`."""
    _on(t, what, dev)
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor expected")
    return t.data_ptr()


def _rows(t, heads: int, d: int, what: str, dev: int):
    """Address and token stride of [n, heads, d] rows on device `dev` whose last two axes are contiguous."""
    _on(t, what, dev)
    n, h, e = t.shape if t.dim() == 3 else (0, 0, 0)
    if h != heads or e != d:
        raise ValueError(f"{what}: [n, {heads}, {d}] expected, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != d):
        raise ValueError(f"{what}: the last two axes must be contiguous")
    return t.data_ptr(), s0 if n > 1 else heads * d


def kv4_block_bytes(page: int, d: int) -> int:
    """Bytes of one (page, key head) block."""
    return _bytes(_c.kv4_block_bytes(page, d), "kv4_block_bytes")


class Kv4:
    """One layer's cache: data uint8 [npages, nkv * kv4_block_bytes(page, d)] (16-byte aligned device memory)."""

    __slots__ = ("data", "page", "nkv", "d", "dev", "c", "ref")

    def __init__(self, data, page: int, nkv: int, d: int):
        per = nkv * kv4_block_bytes(page, d)
        if data.dtype is not torch.uint8 or data.numel() % per:
            raise ValueError(f"data: uint8 pages of {per} bytes expected")
        self.data, self.page, self.nkv, self.d = data, page, nkv, d
        self.dev = _on(data, "data")
        self.c = _CKv4(_dev(data, None, "data", self.dev), data.numel() // per, page, nkv, d)
        self.ref = ctypes.addressof(self.c)


class KvSeqs:
    """The sequences of a call: tables int32 [nrows, maxp], lens int32 [nrows]; rows int32 [nseq] chooses and orders them
    (None: all, in order), q_start int32 [nseq + 1] bounds each one's new tokens (None: one token each)."""

    __slots__ = ("tables", "lens", "rows", "q_start", "dev", "c", "ref")

    def __init__(self, tables, lens, rows=None, q_start=None):
        i32 = torch.int32
        nrows, maxp = tables.shape
        if lens.numel() != nrows:
            raise ValueError("lens: one length a table row expected")
        nseq = nrows if rows is None else rows.numel()
        if q_start is not None and q_start.numel() != nseq + 1:
            raise ValueError("q_start: nseq + 1 entries expected")
        self.tables, self.lens, self.rows, self.q_start = tables, lens, rows, q_start
        self.dev = dev = _on(tables, "tables")
        self.c = _CSeqs(_dev(tables, i32, "tables", dev), _dev(lens, i32, "lens", dev),
                        None if rows is None else _dev(rows, i32, "rows", dev),
                        None if q_start is None else _dev(q_start, i32, "q_start", dev), nrows, maxp, nseq)
        self.ref = ctypes.addressof(self.c)


class KvPages:
    """The state of a pool's pages, all int32 device tensors: nfree [1], free [npages], refs [npages], lens [nrows],
    tables [nrows, maxp]."""

    __slots__ = ("page", "nfree", "free", "refs", "lens", "tables", "dev", "c", "ref")

    def __init__(self, page: int, nfree, free, refs, lens, tables):
        i32 = torch.int32
        nrows, maxp = tables.shape
        npages = refs.numel()
        if free.numel() != npages or lens.numel() != nrows or nfree.numel() != 1:
            raise ValueError("nfree [1], free and refs [npages], lens [nrows], tables [nrows, maxp] expected")
        self.page, self.nfree, self.free, self.refs, self.lens, self.tables = page, nfree, free, refs, lens, tables
        self.dev = dev = _on(refs, "refs")
        self.c = _CPages(_dev(nfree, i32, "nfree", dev), _dev(free, i32, "free", dev), _dev(refs, i32, "refs", dev),
                         _dev(lens, i32, "lens", dev), _dev(tables, i32, "tables", dev), page, npages, nrows, maxp)
        self.ref = ctypes.addressof(self.c)


# ------------------------------------------------------------------ rows and attention

def kv4_append(cache: Kv4, k, v, slots, stream=None) -> None:
    """Writes the rows k, v [n, nkv, d] into the cache at slots int32 [n] (page * cache.page + place; below zero: passed over)."""
    dev = cache.dev
    kp, ks = _rows(k, cache.nkv, cache.d, "k", dev)
    vp, vs = _rows(v, cache.nkv, cache.d, "v", dev)
    if k.dtype is not v.dtype or k.dtype not in _TYPE or k.shape[0] != v.shape[0] or slots.numel() != k.shape[0]:
        raise ValueError("k, v: float32, float16 or bfloat16 rows of one type, one slot each, expected")
    _check(_c.kv4_append(cache.ref, _TYPE[k.dtype], kp, ks, vp, vs, _dev(slots, torch.int32, "slots", dev), k.shape[0],
                         _stream(stream, dev)), "kv4_append")


def kv4_read(cache: Kv4, slots, k, v, stream=None) -> None:
    """Reads the rows at slots int32 [n] back into k, v [n, nkv, d] (any of the three types)."""
    dev = cache.dev
    kp, ks = _rows(k, cache.nkv, cache.d, "k", dev)
    vp, vs = _rows(v, cache.nkv, cache.d, "v", dev)
    if k.dtype is not v.dtype or k.dtype not in _TYPE or k.shape[0] != v.shape[0] or slots.numel() != k.shape[0]:
        raise ValueError("k, v: float32, float16 or bfloat16 rows of one type, one slot each, expected")
    _check(_c.kv4_read(cache.ref, _TYPE[k.dtype], _dev(slots, torch.int32, "slots", dev), k.shape[0], kp, ks, vp, vs,
                       _stream(stream, dev)), "kv4_read")


def kv4_attn_workspace_bytes(cache: Kv4, q, seqs: KvSeqs = None) -> int:
    """Workspace of kv4_attn for queries like q [ntok, nh, d] (any number of tokens and sequences)."""
    return _bytes(_c.kv4_attn_workspace_bytes(cache.ref, q.shape[1]), "kv4_attn_workspace_bytes")


def kv4_attn(cache: Kv4, q, seqs: KvSeqs, scale: float, out, lse=None, window: int = 0, workspace=None,
             stream=None) -> None:
    """Causal attention of the new tokens q [ntok, nh, d] over the cache: out like q, lse f32 [ntok, nh] (optional);
    window > 0: only the last `window` keys.  workspace: uint8, kv4_attn_workspace_bytes long (allocated here when None)."""
    nh, dev = q.shape[1], cache.dev
    if seqs.dev != dev:
        raise ValueError(f"seqs: on cuda:{seqs.dev}, where the cache is on cuda:{dev}")
    qp, qs = _rows(q, nh, cache.d, "q", dev)
    op, os_ = _rows(out, nh, cache.d, "out", dev)
    if q.dtype is not out.dtype or q.dtype not in _TYPE or q.shape[0] != out.shape[0]:
        raise ValueError("q, out: one shape and one of float32, float16, bfloat16 expected")
    lp = None
    if lse is not None:
        lp = _dev(lse, torch.float32, "lse", dev)
        if lse.numel() != q.shape[0] * nh:
            raise ValueError("lse: [ntok, nh] expected")
    if workspace is None:
        workspace = _workspace(kv4_attn_workspace_bytes(cache, q), q, stream)
    _check(_c.kv4_attn(cache.ref, seqs.ref, _TYPE[q.dtype], qp, qs, q.shape[0], nh, scale, window, op, os_, lp,
                       _dev(workspace, None, "workspace", dev), workspace.numel() * workspace.element_size(),
                       _stream(stream, dev)), "kv4_attn")


# ------------------------------------------------------------------ pages

def _pool(data, npages: int, dev: int):
    """Address, layers and page bytes of a pool [layers, npages, ...] (or [npages, ...]: one layer) of any type."""
    layers = data.shape[0] if data.dim() > 2 else 1
    if (data.shape[1] if data.dim() > 2 else data.shape[0]) != npages:
        raise ValueError(f"data: [layers, {npages}, page] expected, got {tuple(data.shape)}")
    return _dev(data, None, "data", dev), layers, data.numel() * data.element_size() // (layers * npages)


def kv_pages_workspace_bytes(pages: KvPages) -> int:
    """Workspace of kv_pages_fork and kv_pages_compact."""
    return _bytes(_c.kv_pages_workspace_bytes(pages.ref), "kv_pages_workspace_bytes")


def _page_ws(pages, workspace, stream):
    if workspace is None:
        workspace = _workspace(kv_pages_workspace_bytes(pages), pages.refs, stream)
    return workspace, workspace.numel() * workspace.element_size()


def kv_pages_reset(pages: KvPages, stream=None) -> None:
    """Every page free, every sequence empty."""
    _check(_c.kv_pages_reset(pages.ref, _stream(stream, pages.dev)), "kv_pages_reset")


def kv_pages_extend(pages: KvPages, rows, counts, slots, status, stream=None) -> None:
    """counts[i] more tokens for sequence rows[i]: takes pages, grows the lengths, writes the new tokens' slots one
    request after another, and status[i] (QB_OK, QB_E_PAGES, QB_E_ARG).  All int32 device tensors."""
    i32, n = torch.int32, rows.numel()
    if counts.numel() != n or status.numel() < n:
        raise ValueError("counts, status: one entry a row expected")
    _check(_c.kv_pages_extend(pages.ref, _dev(rows, i32, "rows", pages.dev), _dev(counts, i32, "counts", pages.dev), n,
                              _dev(slots, i32, "slots", pages.dev), slots.numel(), _dev(status, i32, "status", pages.dev),
                              _stream(stream, pages.dev)), "kv_pages_extend")


def kv_pages_fork(pages: KvPages, data, parents, children, status, workspace=None, stream=None) -> None:
    """Empty sequence children[i] becomes a copy of parents[i]: full pages shared, the partly filled one copied in every
    layer of data [layers, npages, ...]."""
    i32, n = torch.int32, parents.numel()
    if children.numel() != n or status.numel() < n:
        raise ValueError("children, status: one entry a parent expected")
    dp, layers, pb = _pool(data, pages.c.npages, pages.dev)
    ws, wb = _page_ws(pages, workspace, stream)
    _check(_c.kv_pages_fork(pages.ref, dp, layers, pb, _dev(parents, i32, "parents", pages.dev), _dev(children, i32, "children", pages.dev),
                            n, _dev(status, i32, "status", pages.dev), _dev(ws, None, "workspace", pages.dev), wb, _stream(stream, pages.dev)),
           "kv_pages_fork")


def kv_pages_free(pages: KvPages, rows, stream=None) -> None:
    """Sequences rows (int32) become empty; pages nobody holds go back to the stack."""
    _check(_c.kv_pages_free(pages.ref, _dev(rows, torch.int32, "rows", pages.dev), rows.numel(), _stream(stream, pages.dev)),
           "kv_pages_free")


def kv_pages_compact(pages: KvPages, data, workspace=None, stream=None) -> None:
    """Moves the held pages to the pool's beginning, in every layer of data."""
    dp, layers, pb = _pool(data, pages.c.npages, pages.dev)
    ws, wb = _page_ws(pages, workspace, stream)
    _check(_c.kv_pages_compact(pages.ref, dp, layers, pb, _dev(ws, None, "workspace", pages.dev), wb, _stream(stream, pages.dev)),
           "kv_pages_compact")


def kv_pages_copy(data, npages: int, src, dst, stream=None) -> None:
    """Copies pages src[i] to dst[i] (int32) in every layer of data [layers, npages, ...]."""
    n = src.numel()
    if dst.numel() != n:
        raise ValueError("src, dst: as many destinations as sources expected")
    dev = _on(data, "data")
    dp, layers, pb = _pool(data, npages, dev)
    _check(_c.kv_pages_copy(dp, layers, npages, pb, _dev(src, torch.int32, "src", dev),
                            _dev(dst, torch.int32, "dst", dev), n, _stream(stream, dev)), "kv_pages_copy")
