"""Attention over drafted trees and with sinks on the GPU against 64 bits, with the tolerances of test_gpu_kv4.py (the same
kernels' arithmetic; which keys a token sees changes no rounding)."""
import random

import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
import kv4_ref as ref
from test_gpu_kv4 import Batch, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qb.lib()
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


def seen_keys(n, T, j, window, sinks, marks=None):
    """The keys that token j of T new ones of a sequence of n sees; marks: the drafts that it marks, as bits."""
    base = n - T
    if marks is None:
        keys = list(range(max(0, base + j + 1)))
    else:
        keys = list(range(max(0, base))) + [base + i for i in range(T) if marks >> i & 1 and base + i >= 0]
    if window:
        keys = sorted(set(keys[-window:]) | {k for k in keys if k < sinks})
    return keys


def attention(q, k, v, n, T, scale, seen):
    """kv4_ref.attention over the keys seen[j] of each token."""
    nh, d = q.shape[1:]
    out, mag = np.zeros((T, nh, d)), np.zeros((T, nh, d))
    lse, zabs = np.full((T, nh), -np.inf), np.zeros((T, nh))
    for j in range(T):
        if not seen[j]:
            continue
        o, l, z, m = ref.attention(q[j:j + 1], k[seen[j]], v[seen[j]], len(seen[j]), 1, scale, 0)
        out[j], lse[j], zabs[j], mag[j] = o[0], l[0], z[0], m[0]
    return out, lse, zabs, mag


def random_tree(r, T):
    """Parents of a tree whose numbers ascend from parent to child, and each token's marks."""
    parents = [-1] + [r.randrange(max(0, j - 6), j) for j in range(1, T)]
    marks = []
    for j, p in enumerate(parents):
        marks.append((marks[p] if p >= 0 else 0) | 1 << j)
    return parents, marks


class Ext(Batch):
    """A batch with sinks, or trees: marks[s][j] of sequence s."""

    def __init__(self, *a, sinks=0, marks=None, words=None, **kw):
        super().__init__(*a, **kw)
        self.sinks, self.marks = sinks, marks
        if marks is not None:
            words = words or max(1, -(-max(self.news) // 32))
            flat = [[m >> 32 * w & 0xFFFFFFFF for w in range(words)] for s in marks for m in s]
            self.masks = _i32(np.array(flat, np.uint32).reshape(-1, words).view(np.int32))

    def run(self, scale, window=0, rows=None, stream=None, workspace=None):
        import torch
        seqs = qb.KvSeqs(_i32(self.tables), _i32(self.lens), rows=rows, q_start=_i32(self.q_start))
        out = torch.full_like(self.q, 9.0)
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        if self.marks is None:
            qb.kv4_attn_sinks(self.cache, self.q, seqs, scale, out, window, self.sinks, lse=lse, stream=stream, workspace=workspace)
        else:
            qb.kv4_attn_tree(self.cache, self.q, seqs, self.masks, scale, out, lse=lse, window=window, sinks=self.sinks, stream=stream, workspace=workspace)
        torch.cuda.synchronize()
        return out, lse

    def want(self, scale, window=0):
        parts, at = [], 0
        q = self.q.double().cpu().numpy()
        for s, (n, T) in enumerate(zip(self.lens, self.news)):
            a = self.q_start[s]
            seen = [seen_keys(n, T, j, window, self.sinks, None if self.marks is None else self.marks[s][j]) for j in range(T)]
            parts.append(attention(q[a:a + T], self.k[at:at + n], self.v[at:at + n], n, T, scale, seen))
            at += n
        return [np.concatenate(x) for x in zip(*parts)]


def trees(seed, news, kind="tree"):
    r = random.Random(seed)
    if kind == "any":
        return [[r.getrandbits(T) if r.random() < 0.8 else 0 for _ in range(T)] for T in news]
    return [random_tree(r, T)[1] if T else [] for T in news]


HEADS = [(8, 2, 128, 16), (9, 3, 64, 64), (4, 2, 256, 32), (5, 1, 80, 16), (16, 1, 128, 64)]


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (7, 40), (40, 4), (100, 33)])
@pytest.mark.parametrize("nh,nkv,d,page", HEADS)
def test_sinks_steps(name, window, sinks, nh, nkv, d, page):
    """One token and a few a sequence; sequences shorter than the sinks, empty, shorter than their new tokens."""
    lens, news = [0, 1, 3, 16, 33, 40, 64, 130, 200, 257, 300], [1, 1, 5, 1, 2, 0, 3, 1, 4, 1, 2]
    Ext(nh + window, lens, news, nh, nkv, d, page, name, sinks=sinks).check(window=window)


@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(50, 4), (128, 130), (300, 256), (1, 1000)])
@pytest.mark.parametrize("nh,nkv,d,page", [(4, 2, 128, 64), (3, 1, 64, 16)])
def test_sinks_prompts(name, window, sinks, nh, nkv, d, page):
    """Many tokens a sequence (half precision: the tensor-memory kernel): tiles of sinks, a gap, tiles of the window."""
    Ext(window, [700, 129, 400], [300, 129, 260], nh, nkv, d, page, name, sinks=sinks).check(window=window)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_sinks_long_sequences_are_split(name):
    Ext(3, [9001, 40, 7000, 6001], [1, 1, 2, 3], 4, 1, 128, 16, name, sinks=70).check(window=3000)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T", [2, 90])
def test_without_sinks_as_before(name, T):
    """No sinks, or no window: kv4_attn's bits."""
    import torch
    for window, sinks in ((40, 0), (0, 7), (0, 0)):
        b = Ext(4, [300, 170], [T, 40 if T > 40 else 1], 4, 2, 128, 16, name, sinks=sinks)
        got = b.run(0.1, window)
        want = Batch.run(b, 0.1, window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (5, 3), (40, 34)])
@pytest.mark.parametrize("nh,nkv,d,page", HEADS)
def test_trees(name, kind, window, sinks, nh, nkv, d, page):
    """Trees and any marks (empty ones too); sequences that are all drafts, shorter than their drafts, without drafts."""
    lens, news = [40, 8, 5, 70, 0, 130, 64, 33, 300], [5, 8, 9, 35, 2, 33, 0, 1, 17]
    Ext(nh + window, lens, news, nh, nkv, d, page, name, sinks=sinks, marks=trees(window, news, kind)).check(window=window)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 5), (200, 140)])
@pytest.mark.parametrize("nh,nkv,d,page", [(8, 2, 128, 16), (4, 1, 64, 32)])
def test_wide_trees(name, kind, window, sinks, nh, nkv, d, page):
    """Enough rows for the tensor-memory kernel; drafts over three words and tile ends."""
    lens, news = [500, 90, 260, 64, 2500], [70, 90, 40, 64, 33]
    Ext(window + nh, lens, news, nh, nkv, d, page, name, sinks=sinks, marks=trees(window, news, kind)).check(window=window)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 5), (700, 300)])
@pytest.mark.parametrize("nh,nkv,d,page", [(8, 2, 128, 16), (8, 1, 64, 64), (9, 1, 96, 32)])
def test_trees_of_one_row_tile(name, window, sinks, nh, nkv, d, page):
    """Sequences whose rows fill one tile of 128 at the most: one key tile, two, three, many; some with more rows between them."""
    lens, news = [100, 200, 300, 30, 2500, 1000, 129, 128, 5000, 400], [16, 12, 31, 30, 14, 60, 20, 13, 9, 40]
    Ext(window + nh, lens, news, nh, nkv, d, page, name, sinks=sinks, marks=trees(window, news)).check(window=window)


@pytest.mark.parametrize("nkv", [1, 8])
def test_a_row_tile_is_joined_with_other_blocks(nkv):
    """Long sequences with few rows: pieces of an item in several blocks, each of two halves."""
    news = [20, 25, 17]
    Ext(nkv, [6001, 900, 3000], news, 4 * nkv, nkv, 128, 16, "f16", marks=trees(1, news)).check()
    Ext(nkv, [6001, 900, 3000], news, 4 * nkv, nkv, 64, 16, "bf16", sinks=200).check(window=2500)


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_large_steps_in_a_row_tile(name):
    """Steps past 2^12 and steps that are not finite, in values of a sequence of one row tile.  Scores of magnitudes of some 10 and
    values in f16 are off by 2^-11 each at the most, a probability by 2^-11 and as much by its score's: less than 2^-9 of the
    weighed magnitudes together."""
    import torch
    news = [24, 20]
    b = Ext(7, [700, 300], news, 8, 2, 128, 16, name, marks=trees(5, news), sinks=3)
    before = b.run(0.1, 130)
    place = np.array([550, 600])  # of sequence 0: out of the window and in it
    slots = _i32(b.tables[0, place // 16] * 16 + place % 16)
    k, v = torch.zeros((2, 2, 128), device="cuda"), torch.zeros((2, 2, 128), device="cuda")
    v[:, 0, :32] = 50000.0
    v[0, 1] = 1e30
    qb.kv4_append(b.cache, k, v, slots)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    qb.kv4_read(b.cache, slots, kb, vb)
    b.k[place], b.v[place] = kb.double().cpu().numpy(), vb.double().cpu().numpy()
    seen = [seen_keys(700, 24, j, 130, 3, b.marks[0][j]) for j in range(24)]
    out, lse = b.run(0.1, 130)
    assert torch.equal(out[24:], before[0][24:])
    for j in range(24):  # key 550 is seen by the tokens whose path is short
        assert bool(torch.isnan(out[j, 4:]).all()) == (550 in seen[j]) and 600 in seen[j]
        assert not bool(torch.isnan(out[j, :4]).any())
    b.v[550, 1] = 0.0
    want = attention(b.q[:24].double().cpu().numpy(), b.k[:700], b.v[:700], 700, 24, 0.1, seen)
    got = out[:24, :4].double().cpu().numpy()
    assert np.all(np.abs(got - want[0][:, :4]) <= 2.0 ** -9 * want[3][:, :4] + 2.0 ** -8 * np.abs(want[0][:, :4]) + 2.0 ** -24)


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_trees_on_long_sequences_are_split(name):
    news = [7, 1, 12]
    Ext(5, [9001, 40, 5000], news, 4, 1, 128, 16, name, marks=trees(1, news)).check()
    Ext(5, [9001, 40, 5000], news, 4, 1, 128, 16, name, marks=trees(1, news), sinks=50).check(window=4000)


def test_drafts_past_the_words_are_seen_by_none():
    """40 drafts with one word of marks: the last 8 are no one's, not even their own."""
    r = random.Random(2)
    marks = [[r.getrandbits(32) for _ in range(40)]]
    Ext(6, [100], [40], 4, 1, 64, 16, "f32", marks=marks, words=1).check()
    Ext(6, [100], [40], 4, 1, 64, 16, "bf16", marks=marks, words=1).check(window=20)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T", [6, 40])
def test_a_draft_that_is_not_seen_changes_no_bit(name, T):
    """Keys and values of infinite and large steps at drafts, and at keys between sinks and window, that a token does not see."""
    import torch
    news, marks = [T], [[(1 << j) | 1 for j in range(T)]]  # the root and itself
    for window, sinks, spoiled in ((0, 0, [3]), (20, 2, [3]), (20, 2, [3 - 60, 3])):
        b = Ext(9, [200], news, 8, 2, 128, 16, name, marks=marks, sinks=sinks)
        before = b.run(0.1, window)
        for value in (1e30, 60000.0):
            place = np.array([200 - T + x for x in spoiled])
            slots = _i32(b.tables[0, place // 16] * 16 + place % 16)
            x = torch.full((len(place), 2, 128), value, device="cuda")
            qb.kv4_append(b.cache, x, x, slots)
            after = b.run(0.1, window)
            others = [j for j in range(T) if j != 3]
            assert torch.equal(after[0][others], before[0][others]) and torch.equal(after[1][others], before[1][others])
            assert not torch.equal(after[1][3], before[1][3])


def test_a_chain_is_causal():
    """Marks of a chain: kv4_attn's results within its tolerance, with a window too."""
    for name in ("f32", "bf16"):
        for window in (0, 9):
            news = [5, 8, 30, 1]
            b = Ext(2, [40, 8, 130, 64], news, 8, 2, 128, 16, name, marks=[[(2 << j) - 1 for j in range(T)] for T in news])
            b.check(window=window)
            b.marks = None
            b.sinks = 0
            want = Ext.want(b, 0.1, window)
            assert np.allclose(want[1], Batch.want(b, 0.1, window)[1])


def test_places_past_32_bits():
    """A cache of more than 2^32 bytes whose last pages hold the keys."""
    import torch
    nkv, d, page, npages = 8, 128, 64, 60000
    pool = torch.empty((npages, nkv * qb.kv4_block_bytes(page, d)), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 32
    small = Ext(8, [200], [9], 16, nkv, d, page, "f32", marks=trees(3, [9]), sinks=3)
    used = small.tables[0, :4]
    pool[npages - 4:] = small.pool[torch.from_numpy(used).long().cuda()]
    want = small.run(0.1, 50)
    small.tables[0, :4] = np.arange(npages - 4, npages)
    small.cache = qb.Kv4(pool, page, nkv, d)
    got = small.run(0.1, 50)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strides_and_tokens_of_no_sequence():
    """Queries and outputs inside a wider buffer; tokens before the first and behind the last sequence stay as they were."""
    import torch
    news = [4, 3]
    b = Ext(1, [50, 90], news, 4, 2, 64, 16, "bf16", marks=trees(4, news), sinks=2)
    want = b.run(0.1, 20)
    wide = torch.full((7 + 5, 3 * 4 * 64), 5.0, device="cuda", dtype=torch.bfloat16)
    q, out = wide[:, :256].unflatten(1, (4, 64)), wide[:, 512:].unflatten(1, (4, 64))
    q[2:9] = b.q
    masks = torch.full((12, 1), -1, dtype=torch.int32, device="cuda")
    masks[2:9] = b.masks
    lse = torch.full((12, 4), 5.0, device="cuda")
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens), q_start=_i32([2, 6, 9]))
    qb.kv4_attn_tree(b.cache, q, seqs, masks, 0.1, out, lse=lse, window=20, sinks=2)
    assert torch.equal(out[2:9], want[0]) and torch.equal(lse[2:9], want[1])
    assert bool((out[:2] == 5).all()) and bool((out[9:] == 5).all()) and bool((lse[9:] == 5).all()) and bool((wide[:, 256:512] == 5).all())


def test_captured_and_on_another_stream():
    """A call captured into a graph and replayed on changed queries, masks and lengths; two calls at once, each with its workspace."""
    import torch
    news = [6, 40]
    b = Ext(3, [300, 170], news, 8, 2, 128, 16, "bf16", marks=trees(7, news), sinks=4)
    c = Ext(4, [700, 90], [5, 5], 8, 2, 128, 16, "bf16", sinks=4)
    wants = [b.run(0.1, 50), c.run(0.1, 50)]
    work = [torch.empty(qb.kv4_attn_workspace_bytes(x.cache, x.q), dtype=torch.uint8, device="cuda") for x in (b, c)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        outs = [(torch.empty_like(x.q), torch.empty(x.q.shape[:2], device="cuda")) for x in (b, c)]
        seqs = [qb.KvSeqs(_i32(x.tables), _i32(x.lens), q_start=_i32(x.q_start)) for x in (b, c)]
        torch.cuda.synchronize()
        qb.kv4_attn_tree(b.cache, b.q, seqs[0], b.masks, 0.1, outs[0][0], lse=outs[0][1], window=50, sinks=4, workspace=work[0], stream=streams[0])
        qb.kv4_attn_sinks(c.cache, c.q, seqs[1], 0.1, outs[1][0], 50, 4, lse=outs[1][1], workspace=work[1], stream=streams[1])
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, wants):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    out, lse, seqs, masks, q = torch.empty_like(b.q), torch.empty(b.q.shape[:2], device="cuda"), seqs[0], b.masks.clone(), b.q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qb.kv4_attn_tree(b.cache, q, seqs, masks, 0.1, out, lse=lse, window=50, sinks=4, workspace=work[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, wants[0][0]) and torch.equal(lse, wants[0][1])
    b.marks = trees(8, news)
    masks.copy_(_i32(np.array([[m & 0xFFFFFFFF, m >> 32] for s in b.marks for m in s], np.uint32).view(np.int32)))
    q.mul_(-1.5)
    b.q, b.masks = q.clone(), masks
    graph.replay()
    torch.cuda.synchronize()
    replayed = out.clone(), lse.clone()
    want = b.run(0.1, 50)
    assert torch.equal(replayed[0], want[0]) and torch.equal(replayed[1], want[1])
    b.check(0.1, 50)


def test_bad_pages_and_rows_are_reported():
    """A page or row number outside its range reads as page 0 or as no keys, and is reported."""
    import torch
    news = [3, 2]
    b = Ext(1, [50, 90], news, 4, 2, 64, 16, "f32", marks=trees(4, news))
    want = b.run(0.1)
    torch.cuda.synchronize()
    b.tables[1, 2] = 1 << 20
    out, lse = b.run(0.1)
    assert qb.q_device_status() == qb.QB_E_INDEX and qb.q_device_status() == qb.QB_OK
    assert torch.equal(out[:3], want[0][:3])
    b.tables[1, 2] = 0
    out, lse = b.run(0.1, rows=_i32([0, 7]))
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert torch.equal(out[:3], want[0][:3])


def test_refusals():
    import torch
    b = Ext(1, [50], [3], 4, 2, 64, 16, "f32", marks=trees(4, [3]), sinks=1)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens), q_start=_i32(b.q_start))
    out = torch.empty_like(b.q)
    for masks in (b.masks[:2], b.masks.float(), b.masks.cpu(), b.masks[:, 0], torch.zeros((3, 40), dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            qb.kv4_attn_tree(b.cache, b.q, seqs, masks, 0.1, out)
    for masks in (torch.zeros((3, 33), dtype=torch.int32, device="cuda"), torch.zeros((3, 0), dtype=torch.int32, device="cuda")):
        with pytest.raises(qb.QbError):
            qb.kv4_attn_tree(b.cache, b.q, seqs, masks, 0.1, out)
    with pytest.raises(qb.QbError):
        qb.kv4_attn_sinks(b.cache, b.q, seqs, 0.1, out, 4, -1)
    with pytest.raises(qb.QbError):
        qb.kv4_attn_tree(b.cache, b.q, seqs, b.masks, 0.1, out, window=-1)
    empty = torch.empty((0, 4, 64), device="cuda")
    qb.kv4_attn_tree(b.cache, empty, qb.KvSeqs(_i32(b.tables), _i32(b.lens), q_start=_i32([0, 0])), torch.empty((0, 1), dtype=torch.int32, device="cuda"), 0.1, empty)
