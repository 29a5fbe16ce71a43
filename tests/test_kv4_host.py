"""The paged 4-bit cache on a host without a GPU: sizes, argument checks that
answer before any CUDA call, the binding's refusals, and the plain reference's
own layout."""
import ctypes

import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
import kv4_ref as ref
from block_quantized_weight_quantize_gb300 import kv4

A, ODD = 4096, 4098  # never dereferenced: every call fails its checks first


def _cache(**kw):
    a = dict(data=A, npages=8, page=16, nkv=2, d=64)
    a.update(kw)
    return kv4._CKv4(a["data"], a["npages"], a["page"], a["nkv"], a["d"])


def _seqs(**kw):
    a = dict(tables=A, lens=A, rows=None, q_start=None, nrows=4, maxp=4, nseq=3)
    a.update(kw)
    return kv4._CSeqs(*[a[n] for n in ("tables", "lens", "rows", "q_start", "nrows", "maxp", "nseq")])


def _pages(**kw):
    a = dict(nfree=A, free_pages=A, refs=A, lens=A, tables=A, page=16, npages=8, nrows=4, maxp=4)
    a.update(kw)
    return kv4._CPages(*[a[n] for n, _ in kv4._CPages._fields_])


def test_block_bytes():
    for page in (16, 32, 64):
        for d in (8, 64, 72, 128, 136, 256):
            assert qb.kv4_block_bytes(page, d) == ref.block_bytes(page, d)
    for page, d in ((8, 64), (48, 64), (16, 0), (16, 12), (16, 264)):
        assert kv4._c.kv4_block_bytes(page, d) == qb.QB_E_ARG
        with pytest.raises(qb.QbError):
            qb.kv4_block_bytes(page, d)


def test_every_nibble_has_one_place():
    for page in (16, 32, 64):
        for dp in (64, 128, 256):
            r, i = np.arange(page)[:, None], np.arange(dp)[None, :]
            for f in (ref.key_nibble, ref.value_nibble):
                assert sorted(f(page, dp, r, i).flatten().tolist()) == list(range(page * dp))


@pytest.mark.parametrize("bad", [dict(data=None), dict(data=ODD), dict(page=24), dict(npages=0), dict(nkv=0), dict(nkv=2000), dict(d=60), dict(d=512),
                                 dict(npages=1 << 27, page=16)])
def test_bad_caches(bad):
    c = ctypes.addressof(k := _cache(**bad))
    s = ctypes.addressof(t := _seqs())
    assert kv4._c.kv4_append(c, 0, A, 128, A, 128, A, 1, None) == qb.QB_E_ARG
    assert kv4._c.kv4_read(c, 0, A, 1, A, 128, A, 128, None) == qb.QB_E_ARG
    assert kv4._c.kv4_attn(c, s, 0, A, 256, 3, 4, 1.0, 0, A, 256, None, A, 1 << 30, None) == qb.QB_E_ARG
    assert k is not None and t is not None


def test_row_arguments():
    c = ctypes.addressof(k := _cache())

    def append(type_=0, k_=A, ks=128, v=A, vs=128, slots=A, n=3):
        return kv4._c.kv4_append(c, type_, k_, ks, v, vs, slots, n, None)

    assert append(n=0) == qb.QB_OK
    for bad in (dict(type_=3), dict(k_=None), dict(k_=ODD), dict(ks=127), dict(ks=130), dict(v=None), dict(vs=64), dict(slots=None), dict(slots=4097),
                dict(n=-1), dict(n=1 << 31)):
        assert append(**bad) == qb.QB_E_ARG
    assert append(type_=1, ks=132) == qb.QB_E_ARG   # 264 bytes between half-precision rows
    assert kv4._c.kv4_read(c, 0, A, -1, A, 128, A, 128, None) == qb.QB_E_ARG
    assert kv4._c.kv4_read(c, 0, A, 0, A, 128, A, 128, None) == qb.QB_OK
    assert k is not None


def test_attention_arguments():
    c = ctypes.addressof(k := _cache())
    need = kv4._c.kv4_attn_workspace_bytes(c, 4)
    assert need > 0
    keep = []

    def attn(seqs=None, type_=0, q=A, qs=256, ntok=3, nh=4, scale=1.0, window=0, out=A, os_=256, lse=None, ws=A, wb=need):
        keep.append(s := _seqs(**(seqs or {})))
        return kv4._c.kv4_attn(c, ctypes.addressof(s), type_, q, qs, ntok, nh, scale, window, out, os_, lse, ws, wb, None)

    assert attn(seqs=dict(q_start=A), ntok=0) == qb.QB_OK
    for bad in (dict(type_=5), dict(q=None), dict(q=ODD), dict(qs=255), dict(qs=258), dict(ntok=-1), dict(ntok=4), dict(nh=3), dict(nh=0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(window=-1), dict(out=None), dict(os_=8), dict(lse=4097), dict(ws=None),
                dict(ws=ODD), dict(wb=need - 1), dict(seqs=dict(tables=None)), dict(seqs=dict(lens=None)), dict(seqs=dict(nseq=0)),
                dict(seqs=dict(nseq=5)), dict(seqs=dict(maxp=0)), dict(seqs=dict(nseq=9000, rows=A)), dict(seqs=dict(rows=4097))):
        assert attn(**bad) == qb.QB_E_ARG, bad
    assert kv4._c.kv4_attn_workspace_bytes(c, 3) == qb.QB_E_ARG
    assert k is not None


def test_attention_refuses_more_rows_than_an_int_counts():
    c = ctypes.addressof(k := _cache())
    s = _seqs(q_start=A)
    need = kv4._c.kv4_attn_workspace_bytes(c, 4096)
    assert need > 0
    for ntok, nh in ((1 << 24, 128), ((1 << 24) + 1, 4), (1 << 19, 4096)):
        assert kv4._c.kv4_attn(c, ctypes.addressof(s), 0, A, nh * 64, ntok, nh, 1.0, 0, A, nh * 64, None, A, need, None) == qb.QB_E_ARG
    assert k is not None


def test_page_arguments():
    good = _pages()
    p = ctypes.addressof(good)
    ws = kv4._c.kv_pages_workspace_bytes(p)
    assert ws > 0
    for bad in (dict(nfree=None), dict(free_pages=None), dict(refs=None), dict(lens=None), dict(tables=None), dict(tables=4097), dict(page=20),
                dict(npages=0), dict(npages=(1 << 20) + 1), dict(nrows=0), dict(maxp=0)):
        b = _pages(**bad)
        a = ctypes.addressof(b)
        assert kv4._c.kv_pages_workspace_bytes(a) == qb.QB_E_ARG
        assert kv4._c.kv_pages_reset(a, None) == qb.QB_E_ARG
        assert kv4._c.kv_pages_free(a, A, 1, None) == qb.QB_E_ARG
        assert kv4._c.kv_pages_extend(a, A, A, 1, A, 1, A, None) == qb.QB_E_ARG
        assert kv4._c.kv_pages_fork(a, A, 1, 64, A, A, 1, A, A, 1 << 20, None) == qb.QB_E_ARG
        assert kv4._c.kv_pages_compact(a, A, 1, 64, A, 1 << 20, None) == qb.QB_E_ARG
    f = kv4._c
    assert f.kv_pages_free(p, None, 1, None) == qb.QB_E_ARG and f.kv_pages_free(p, A, 5, None) == qb.QB_E_ARG
    assert f.kv_pages_free(p, A, 0, None) == qb.QB_OK
    assert f.kv_pages_extend(p, A, None, 1, A, 1, A, None) == qb.QB_E_ARG and f.kv_pages_extend(p, A, A, 0, A, 1, A, None) == qb.QB_OK
    assert f.kv_pages_fork(p, A, 1, 60, A, A, 1, A, A, ws, None) == qb.QB_E_ARG     # page bytes
    assert f.kv_pages_fork(p, ODD, 1, 64, A, A, 1, A, A, ws, None) == qb.QB_E_ARG
    assert f.kv_pages_fork(p, A, 0, 64, A, A, 1, A, A, ws, None) == qb.QB_E_ARG     # layers
    assert f.kv_pages_fork(p, A, 1, 64, A, A, 1, A, A, ws - 1, None) == qb.QB_E_ARG
    assert f.kv_pages_fork(p, A, 1, 64, A, A, 0, A, A, ws, None) == qb.QB_OK
    assert f.kv_pages_compact(p, A, 1, 64, None, ws, None) == qb.QB_E_ARG
    assert f.kv_pages_copy(A, 1, 8, 64, A, A, 9, None) == qb.QB_E_ARG and f.kv_pages_copy(A, 1, 8, 64, None, A, 1, None) == qb.QB_E_ARG
    assert f.kv_pages_copy(A, 1, 8, 64, A, A, 0, None) == qb.QB_OK


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    with pytest.raises(ValueError):
        qb.Kv4(torch.zeros((2, qb.kv4_block_bytes(16, 64)), dtype=torch.uint8), 16, 1, 64)
    with pytest.raises(ValueError):
        qb.Kv4(torch.zeros((2, 100), dtype=torch.uint8), 16, 1, 64)
    with pytest.raises(ValueError):
        qb.KvSeqs(torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        qb.KvSeqs(torch.zeros((2, 3), dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        qb.KvPages(16, *(torch.zeros(s, dtype=torch.int32) for s in (1, 4, 4, 2, (2, 3))))
    with pytest.raises(AttributeError):
        qb.kv4_nothing


def test_status_texts():
    assert "page" in qb.strerror(qb.QB_E_PAGES) and "outside" in qb.strerror(qb.QB_E_INDEX)
