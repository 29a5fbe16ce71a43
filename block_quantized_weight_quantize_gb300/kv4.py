"""Binding of the paged 4-bit key/value cache: rows in and out, attention over
it, and its pages (``kv4_*`` and ``kv_pages_*`` of ``include/qgemv.h``); drafted
trees over it (``kv_tree_*``) and log probabilities (``q_logprobs``).

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
    "kv4_attn_sinks": ([_P, _P, _I, _P, _L, _L, _I, ctypes.c_float, _I, _I, _P, _L, _P, _P, ctypes.c_size_t, _P], _I),
    "kv4_attn_tree": ([_P, _P, _I, _P, _L, _L, _I, ctypes.c_float, _I, _I, _P, _I, _P, _L, _P, _P, ctypes.c_size_t, _P], _I),
    "kv_tree_masks": ([_P, _L, _P, _I, _P, _I, _P, _P], _I),
    "kv_tree_accept": ([_P, _P, _P, _L, _P, _I, _P, _P, _P, _P], _I),
    "q_logprobs": ([_I, _P, _L, _L, _L, ctypes.c_float, _P, _I, _P, _P, _P, _I, _P, _P, _P], _I),
    "kv4_keep": ([_P, _P, _I, _I, _I, _P, _P, _P, _P, _L, _I, _P, _P], _I),
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
    if t.get_device() != dev:
        _on(t, what, dev)
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous tensor expected")
    return t.data_ptr()


def _rows(t, heads: int, d: int, what: str, dev: int):
    """Address and token stride of [n, heads, d] rows on device `dev` whose last two axes are contiguous."""
    if t.get_device() != dev:
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


def _attn(call, more, cache: Kv4, q, seqs: KvSeqs, scale, window, out, lse, workspace, stream, where: str) -> None:
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
    _check(call(cache.ref, seqs.ref, _TYPE[q.dtype], qp, qs, q.shape[0], nh, scale, window, *more, op, os_, lp,
                _dev(workspace, None, "workspace", dev), workspace.numel() * workspace.element_size(),
                _stream(stream, dev)), where)


def kv4_attn(cache: Kv4, q, seqs: KvSeqs, scale: float, out, lse=None, window: int = 0, workspace=None,
             stream=None) -> None:
    """Causal attention of the new tokens q [ntok, nh, d] over the cache: out like q, lse f32 [ntok, nh] (optional);
    window > 0: only the last `window` keys.  workspace: uint8, kv4_attn_workspace_bytes long (allocated here when None)."""
    _attn(_c.kv4_attn, (), cache, q, seqs, scale, window, out, lse, workspace, stream, "kv4_attn")


def kv4_attn_sinks(cache: Kv4, q, seqs: KvSeqs, scale: float, out, window: int, sinks: int, lse=None, workspace=None,
                   stream=None) -> None:
    """kv4_attn where a token sees the last `window` keys and, of those before them, the sequence's first `sinks`."""
    _attn(_c.kv4_attn_sinks, (sinks,), cache, q, seqs, scale, window, out, lse, workspace, stream, "kv4_attn_sinks")


def kv4_attn_tree(cache: Kv4, q, seqs: KvSeqs, masks, scale: float, out, lse=None, window: int = 0, sinks: int = 0,
                  workspace=None, stream=None) -> None:
    """kv4_attn over drafted trees: masks int32 [ntok, words], bit i % 32 of word i / 32: the token sees draft i of its
    sequence (kv_tree_masks); a token's window is over the keys before the drafts and its marked drafts."""
    if masks.dim() != 2 or masks.shape[0] != q.shape[0]:
        raise ValueError("masks: [ntok, words] expected")
    more = (sinks, _dev(masks, torch.int32, "masks", cache.dev), masks.shape[1])
    _attn(_c.kv4_attn_tree, more, cache, q, seqs, scale, window, out, lse, workspace, stream, "kv4_attn_tree")


# ------------------------------------------------------------------ drafted trees, log probabilities

def _tree(parents, q_start):
    """Device, tokens, address of q_start and sequences of a tree call."""
    n, dev = parents.numel(), _on(parents, "parents")
    if q_start is None:
        return dev, n, None, n
    if q_start.numel() < 1:
        raise ValueError("q_start: nseq + 1 entries expected")
    return dev, n, _dev(q_start, torch.int32, "q_start", dev), q_start.numel() - 1


def kv_tree_masks(parents, masks, depth=None, q_start=None, stream=None) -> None:
    """parents int32 [ntok] (the number of the draft that a token follows, within its sequence; -1: none) -> masks int32
    [ntok, words] for kv4_attn_tree and depth int32 [ntok] (optional); q_start int32 [nseq + 1] bounds the sequences."""
    i32, (dev, n, sp, nseq) = torch.int32, _tree(parents, q_start)
    if masks.dim() != 2 or masks.shape[0] != n or (depth is not None and depth.numel() != n):
        raise ValueError("masks [ntok, words], depth [ntok] expected")
    _check(_c.kv_tree_masks(_dev(parents, i32, "parents", dev), n, sp, nseq, _dev(masks, i32, "masks", dev), masks.shape[1],
                            None if depth is None else _dev(depth, i32, "depth", dev), _stream(stream, dev)), "kv_tree_masks")


def kv_tree_accept(parents, tokens, targets, keep, nkeep, next, q_start=None, stream=None) -> None:
    """The path that the target's choices take through each tree: keep int32 [ntok] (accepted drafts' numbers, then -1),
    nkeep and next int32 [nseq] (how many, and the target's token after the last)."""
    i32, (dev, n, sp, nseq) = torch.int32, _tree(parents, q_start)
    if tokens.numel() != n or targets.numel() != n or keep.numel() != n or nkeep.numel() != nseq or next.numel() != nseq:
        raise ValueError("tokens, targets, keep [ntok], nkeep, next [nseq] expected")
    _check(_c.kv_tree_accept(_dev(parents, i32, "parents", dev), _dev(tokens, i32, "tokens", dev), _dev(targets, i32, "targets", dev),
                             n, sp, nseq, _dev(keep, i32, "keep", dev), _dev(nkeep, i32, "nkeep", dev), _dev(next, i32, "next", dev),
                             _stream(stream, dev)), "kv_tree_accept")


def q_logprobs(logits, tokens=None, scale: float = 1.0, logprobs=None, entropy=None, lse=None, top_tokens=None, top_logprobs=None,
               stream=None) -> None:
    """From logits [n, vocab] (float32, float16 or bfloat16; rows contiguous) times `scale`: logprobs f32 [n, m] of tokens
    int32 [n, m], entropy and lse f32 [n], the k largest logits' places top_tokens int32 [n, k] and log probabilities
    top_logprobs f32 [n, k].  What is None is not computed."""
    f32, dev, typ = torch.float32, logits.get_device(), _TYPE.get(logits.dtype)
    if dev < 0:
        _on(logits, "logits")
    if logits.dim() != 2 or typ is None:
        raise ValueError("logits: float32, float16 or bfloat16 [n, vocab] expected")
    n, vocab = logits.shape
    stride, one = logits.stride()
    if one != 1 and vocab != 1:
        raise ValueError("logits: contiguous rows expected")
    m = k = 0
    tp = lp = ep = sp = ttp = tlp = None
    if tokens is not None:
        if logprobs is None or tokens.dim() != 2 or tokens.shape[0] != n or logprobs.shape != tokens.shape:
            raise ValueError("tokens and logprobs: [n, m] expected")
        m, tp, lp = tokens.shape[1], _dev(tokens, torch.int32, "tokens", dev), _dev(logprobs, f32, "logprobs", dev)
    elif logprobs is not None:
        raise ValueError("logprobs: of which tokens?")
    if entropy is not None:
        ep = _dev(entropy, f32, "entropy", dev)
        if entropy.numel() != n:
            raise ValueError("entropy: [n] expected")
    if lse is not None:
        sp = _dev(lse, f32, "lse", dev)
        if lse.numel() != n:
            raise ValueError("lse: [n] expected")
    if top_tokens is not None:
        if top_tokens.dim() != 2 or top_tokens.shape[0] != n:
            raise ValueError("top_tokens: [n, k] expected")
        k, ttp = top_tokens.shape[1], _dev(top_tokens, torch.int32, "top_tokens", dev)
    if top_logprobs is not None:
        if top_logprobs.dim() != 2 or top_logprobs.shape[0] != n or (ttp is not None and top_logprobs.shape[1] != k):
            raise ValueError("top_logprobs: [n, k] expected, with top_tokens' k")
        k, tlp = top_logprobs.shape[1], _dev(top_logprobs, f32, "top_logprobs", dev)
    _check(_c.q_logprobs(typ, logits.data_ptr(), stride if n > 1 else vocab, n, vocab, scale, tp, m, lp, ep, sp, k, ttp, tlp,
                         _stream(stream, dev)), "q_logprobs")



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


def kv4_keep(pages: KvPages, data, nkv: int, d: int, rows, q_start, keep, nkeep, status, stream=None) -> None:
    """Of sequence rows[i]'s last q_start[i + 1] - q_start[i] tokens those numbered keep[q_start[i]:][:nkeep[i]] (ascending)
    stay: their rows in every layer of data [layers, npages, ...] (4-bit caches of nkv heads of d) move together, the length
    is lowered, pages past it are given back.  rows None: sequence i.  All int32 device tensors (kv_tree_accept's)."""
    i32, n, dev = torch.int32, nkeep.numel(), pages.dev
    if q_start.numel() != n + 1 or status.numel() < n or (rows is not None and rows.numel() != n):
        raise ValueError("rows, nkeep, status: one entry a request, q_start one more, expected")
    dp, layers, pb = _pool(data, pages.c.npages, dev)
    if pb != nkv * kv4_block_bytes(pages.page, d):
        raise ValueError(f"data: pages of {nkv * kv4_block_bytes(pages.page, d)} bytes expected, got {pb}")
    _check(_c.kv4_keep(pages.ref, dp, layers, nkv, d, None if rows is None else _dev(rows, i32, "rows", dev),
                       _dev(q_start, i32, "q_start", dev), _dev(keep, i32, "keep", dev), _dev(nkeep, i32, "nkeep", dev), keep.numel(), n,
                       _dev(status, i32, "status", dev), _stream(stream, dev)), "kv4_keep")


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
