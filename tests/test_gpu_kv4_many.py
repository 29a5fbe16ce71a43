"""The 4-bit cache's attention over many keys and many sequences, and every call between guard bytes.  Batch and its
tolerances are those of test_gpu_kv4.py."""
import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
from test_gpu_kv4 import Batch, _i32, _type

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("nh,nkv,d,page,window", [(4, 2, 64, 16, 0), (4, 1, 128, 64, 0), (3, 1, 96, 32, 2100)])
def test_prompts_over_many_keys(name, nh, nkv, d, page, window):
    """Row pairs that see fewer and more than 2048 keys follow one another in a block's share, and pieces of both kinds
    are joined; a chunk of sequences with more row pairs than lanes would count by themselves."""
    Batch(nh + d, [5000, 2300, 700, 2100], [300, 600, 100, 2100], nh, nkv, d, page, name).check(window=window)


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_one_prompt_by_itself(name):
    Batch(41, [2304], [2304], 2, 1, 64, 16, name).check()


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts_of_seventy_sequences(name, d):
    """Three chunks of sequences: empty ones, ones without new tokens, ones with more tokens than their cache, one much longer."""
    rng = np.random.default_rng(43)
    lens = [int(x) for x in rng.integers(0, 260, 70)]
    news = [int(rng.integers(0, 200)) if i % 7 else 0 for i in range(70)]
    lens[65], news[65] = 1500, 900
    Batch(43, lens, news, 4, 2, d, 16, name).check()


def _guarded(nbytes, fill):
    """A uint8 buffer of nbytes between 256 guard bytes on each side, and a check that the guards stand."""
    import torch
    whole = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    inner = whole[256:256 + nbytes]
    inner.fill_(fill)

    def stands():
        return bool((whole[:256] == 0xA5).all()) and bool((whole[256 + nbytes:] == 0xA5).all())

    return inner, stands


@pytest.mark.parametrize("name,nh,nkv,d,page,lens,news", [
    ("f32", 4, 2, 64, 16, [37, 0, 300], [1, 1, 1]), ("f32", 7, 1, 128, 32, [900, 33, 5], [5, 3, 1]),
    ("f16", 8, 1, 256, 64, [700, 64], [1, 9]), ("bf16", 9, 3, 72, 16, [2000, 17, 1], [4, 2, 1]),
    ("bf16", 4, 2, 64, 16, [700, 333], [500, 333]), ("f16", 4, 1, 128, 64, [2600, 129, 40], [300, 129, 77])])
def test_nothing_is_written_outside(name, nh, nkv, d, page, lens, news):
    """Rows, outputs, lse and workspace between guard bytes: the guards stand and the results are those of plain buffers."""
    import torch
    b = Batch(51, lens, news, nh, nkv, d, page, name)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(lens), q_start=_i32(b.q_start))
    want, wlse = b.run(0.1)
    es, ntok = b.q.element_size(), sum(news)
    out, out_ok = _guarded(b.q.numel() * es, 0)
    lse, lse_ok = _guarded(ntok * nh * 4, 0)
    work, work_ok = _guarded(qb.kv4_attn_workspace_bytes(b.cache, b.q), 0xFF)
    o, s = out.view(_type(name)).view(b.q.shape), lse.view(torch.float32).view(ntok, nh)
    qb.kv4_attn(b.cache, b.q, seqs, 0.1, o, lse=s, workspace=work)
    assert torch.equal(o, want) and torch.equal(s, wlse)
    assert out_ok() and lse_ok() and work_ok()
    # the rows in and out, the first and last places of the pool among them
    pool, pool_ok = _guarded(b.pool.numel(), 0)
    cache = qb.Kv4(pool.view(b.pool.shape), page, nkv, d)
    n = 2 * page
    slots = _i32(np.concatenate([np.arange(page), b.pool.shape[0] * page - 1 - np.arange(page)]))
    k, v = (torch.randn((n, nkv, d), device="cuda").to(_type(name)) for _ in range(2))
    qb.kv4_append(cache, k, v, slots)
    kb, kb_ok = _guarded(k.numel() * es, 0)
    vb, vb_ok = _guarded(k.numel() * es, 0)
    qb.kv4_read(cache, slots, kb.view(_type(name)).view(k.shape), vb.view(_type(name)).view(k.shape))
    assert pool_ok() and kb_ok() and vb_ok()
    step = 2.0 ** -3 + (2.0 ** -8 if name == "bf16" else 2.0 ** -10)  # half a step of 1/8 at most, the extreme's other side whole
    top = k.float().abs().max()
    assert (kb.view(_type(name)).view(k.shape).float() - k.float()).abs().max() <= top * step


def test_pages_write_nothing_outside():
    import torch
    page, npages, nrows, maxp, layers, words = 16, 37, 9, 5, 3, 12
    sizes = (1, npages, npages, nrows, nrows * maxp)
    state = [_guarded(4 * n, 0) for n in sizes]
    views = [x.view(torch.int32) for x, _ in state]
    views[4] = views[4].view(nrows, maxp)
    pages = qb.KvPages(page, *views)
    data, data_ok = _guarded(layers * npages * words * 4, 0)
    pool = data.view(layers, npages, words * 4)
    work, work_ok = _guarded(qb.kv_pages_workspace_bytes(pages), 0xFF)
    slots, slots_ok = _guarded(4 * 500, 0)
    status, status_ok = _guarded(4 * nrows, 0)
    st = status.view(torch.int32)
    qb.kv_pages_reset(pages)
    qb.kv_pages_extend(pages, _i32(range(6)), _i32([80, 17, 1, 64, 0, 100]), slots.view(torch.int32), st)
    qb.kv_pages_fork(pages, pool, _i32([0, 1, 2]), _i32([6, 7, 8]), st, work)
    qb.kv_pages_free(pages, _i32([0, 3]))
    qb.kv_pages_compact(pages, pool, work)
    qb.kv_pages_copy(pool, npages, _i32([0, 1]), _i32([npages - 1, npages - 2]))
    assert all(ok() for _, ok in state) and data_ok() and work_ok() and slots_ok() and status_ok()
