"""Drafted trees on the GPU: masks and depths, the accepted path, and the kept drafts' rows, lengths and pages, all against lists."""
import random

import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
import kv4_ref as ref
from test_gpu_kv4 import _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qb.lib()
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


def _zeros(*shape):
    import torch
    return torch.full(shape, 77, dtype=torch.int32, device="cuda")


def _starts(news):
    return _i32(np.concatenate([[0], np.cumsum(news)]))


def tree(r, T, kind):
    if T == 0:
        return []
    if kind == "chain":
        return list(range(-1, T - 1))
    if kind == "star":
        return [-1] + [0] * (T - 1)
    if kind == "forest":
        return [r.randrange(-1, j) for j in range(T)]
    return [-1] + [r.randrange(max(0, j - 5), j) for j in range(1, T)]


@pytest.mark.parametrize("kind", ["chain", "star", "forest", "tree"])
@pytest.mark.parametrize("news,words", [([1], 1), ([5, 0, 32, 33], 2), ([64, 1, 31, 0, 100], 4), ([1500, 3], 32), ([40, 70], 1)])
def test_masks_and_depths(kind, news, words):
    r = random.Random(words)
    trees = [tree(r, T, kind) for T in news]
    masks, depth = _zeros(sum(news), words), _zeros(sum(news))
    qb.kv_tree_masks(_i32(sum(trees, [])), masks, depth, q_start=_starts(news))
    want, deep = [], []
    for parents in trees:
        m, d = [], []
        for j, p in enumerate(parents):
            m.append((m[p] if p >= 0 else 0) | 1 << j)
            d.append(d[p] + 1 if p >= 0 else 0)
        want += [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in m]
        deep += d
    assert np.array_equal(masks.cpu().numpy().view(np.uint32), np.array(want, np.uint32).reshape(-1, words))
    assert depth.tolist() == deep
    again = _zeros(sum(news), words)
    qb.kv_tree_masks(_i32(sum(trees, [])), again, q_start=_starts(news))
    assert bool((again == masks).all())


def test_a_long_chain():
    """200000 drafts one after the other, then the path along all of them: a matter of milliseconds."""
    import torch
    T = 200000
    parents = torch.arange(-1, T - 1, dtype=torch.int32, device="cuda")
    masks, depth, start = _zeros(T, 2), _zeros(T), _i32([0, T])
    qb.kv_tree_masks(parents, masks, depth, q_start=start)
    at = torch.arange(T, device="cuda")
    assert torch.equal(depth, at.int())
    want = torch.stack([((1 << (at + 1 - 32 * w).clamp(0, 32)) - 1) for w in (0, 1)], 1)
    assert torch.equal(masks.long() & 0xFFFFFFFF, want)
    keep, nkeep, nxt, ones = _zeros(T), _zeros(1), _zeros(1), torch.ones(T, dtype=torch.int32, device="cuda")
    qb.kv_tree_accept(parents, ones, ones, keep, nkeep, nxt, q_start=start)
    assert torch.equal(keep, at.int()) and nkeep.tolist() == [T] and nxt.tolist() == [1]


def test_masks_of_single_tokens_and_bad_parents():
    masks, depth = _zeros(3, 2), _zeros(3)
    qb.kv_tree_masks(_i32([-1, -1, -1]), masks, depth)
    assert masks.tolist() == [[1, 0]] * 3 and depth.tolist() == [0] * 3
    masks, depth = _zeros(4, 1), _zeros(4)
    qb.kv_tree_masks(_i32([-1, 1, 5, -7]), masks, depth, q_start=_i32([0, 4]))
    assert qb.q_device_status() == qb.QB_E_INDEX and qb.q_device_status() == qb.QB_OK
    assert masks[:, 0].tolist() == [1, 2, 4, 8] and depth.tolist() == [0] * 4
    # bounds outside the tokens are cut to them
    masks = _zeros(4, 1)
    qb.kv_tree_masks(_i32([-1, 0, -1, 0]), masks, q_start=_i32([-5, 2, 9]))
    assert masks[:, 0].tolist() == [1, 3, 1, 3]


def walk(parents, tokens, targets):
    if not parents:
        return [], -1
    path = [0]
    while True:
        nxt = [j for j in range(path[-1] + 1, len(parents)) if parents[j] == path[-1] and tokens[j] == targets[path[-1]]]
        if not nxt:
            return path, targets[path[-1]]
        path.append(nxt[0])


@pytest.mark.parametrize("kind", ["chain", "star", "forest", "tree"])
@pytest.mark.parametrize("news", [[1], [5, 0, 32, 33, 7], [64, 1, 31, 0, 100, 9, 3, 2], [1500, 3]])
def test_accepted_paths(kind, news):
    """Few different tokens, so that paths are long and siblings have the same token."""
    r = random.Random(len(news))
    trees = [tree(r, T, kind) for T in news]
    alphabet = 1 if kind == "chain" else 2
    tokens = [[r.randrange(alphabet) for _ in range(T)] for T in news]
    targets = [[r.randrange(alphabet) for _ in range(T)] for T in news]
    keep, nkeep, nxt = _zeros(sum(news)), _zeros(len(news)), _zeros(len(news))
    qb.kv_tree_accept(*(_i32(sum(x, [])) for x in (trees, tokens, targets)), keep, nkeep, nxt, q_start=_starts(news))
    want = [walk(*x) for x in zip(trees, tokens, targets)]
    assert nkeep.tolist() == [len(p) for p, _ in want] and nxt.tolist() == [t for _, t in want]
    assert keep.tolist() == sum([p + [-1] * (T - len(p)) for (p, _), T in zip(want, news)], [])


class Pool:
    """Sequences in a pool of random bytes, and the same with lists."""

    def __init__(self, seed, lens, page, nkv, d, layers=3, spare=5, shared=()):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.nkv, self.d = list(lens), page, nkv, d
        need = [-(-n // page) for n in lens]
        self.npages = sum(need) + spare
        ids = rng.permutation(self.npages).tolist()
        self.rows, at = [], 0
        for n in need:
            self.rows.append(ids[at:at + n])
            at += n
        self.free = ids[at:]
        self.refs = [0] * self.npages
        for row in self.rows:
            for x in row:
                self.refs[x] += 1
        for x in shared:
            self.refs[self.rows[x[0]][x[1]]] += 1
        self.maxp = max(need) + 1
        self.pool = rng.integers(0, 256, (layers, self.npages, nkv * ref.block_bytes(page, d)), dtype=np.uint8)
        self.dev = torch.from_numpy(self.pool).cuda()
        self.pages = qb.KvPages(page, _i32([len(self.free)]), _i32(self.free + [-1] * (self.npages - len(self.free))), _i32(self.refs), _i32(self.lens),
                                _i32([r + [-1] * (self.maxp - len(r)) for r in self.rows]))

    def row_places(self, slot):
        """Byte numbers within a page of a row's codes, two elements each in their order, and of its steps."""
        page, dp = self.page, ref.padded(self.d)
        r, bb, cb, sb = slot % page, ref.block_bytes(page, self.d), page * dp // 2, page * dp // 16
        i = np.arange(0, dp, 2)
        parts = []
        for h in range(self.nkv):
            for at, nib in ((0, ref.key_nibble(page, dp, r, i)), (cb + sb, ref.value_nibble(page, dp, r, i))):
                parts += [h * bb + at + nib // 2, h * bb + at + cb + r * (dp // 16) + np.arange(dp // 16)]
        return np.concatenate(parts)

    def slot(self, row, place):
        return self.rows[row][place // self.page] * self.page + place % self.page

    def keep(self, row, T, kept):
        base = self.lens[row] - T
        moves = [(self.slot(row, base + j), self.slot(row, base + k)) for k, j in enumerate(kept)]
        held = [self.pool[:, a // self.page, self.row_places(a)].copy() for a, _ in moves]
        for (_, b), x in zip(moves, held):
            self.pool[:, b // self.page, self.row_places(b)] = x
        self.lens[row] = base + len(kept)
        left = -(-self.lens[row] // self.page)
        gone = self.rows[row][left:]
        self.rows[row] = self.rows[row][:left]
        return gone

    def keep_all(self, rows, news, kepts, refused=()):
        back = []
        for i, (row, T, kept) in enumerate(zip(rows, news, kepts)):
            if i in refused:
                continue
            for x in self.keep(row, T, kept):
                self.refs[x] -= 1
                if self.refs[x] == 0:
                    back.append(x)
        self.free += sorted(back)

    def same(self):
        p = self.pages
        assert p.lens.tolist() == self.lens
        assert p.tables.tolist() == [r + [-1] * (self.maxp - len(r)) for r in self.rows]
        assert p.refs.tolist() == self.refs
        assert int(p.nfree) == len(self.free) and p.free[:len(self.free)].tolist() == self.free
        assert np.array_equal(self.dev.cpu().numpy(), self.pool)


def _call(pool, rows, news, kepts, keep=None, nkeep=None):
    flat = keep if keep is not None else sum([k + [-1] * (T - len(k)) for k, T in zip(kepts, news)], [])
    status = _zeros(len(news))
    qb.kv4_keep(pool.pages, pool.dev, pool.nkv, pool.d, None if rows is None else _i32(rows), _starts(news), _i32(flat), _i32(nkeep or [len(k) for k in kepts]), status)
    return status.tolist()


@pytest.mark.parametrize("d,nkv,page", [(64, 3, 16), (128, 8, 16), (128, 1, 64), (256, 2, 32), (8, 1, 64), (80, 2, 32), (136, 1, 16)])
@pytest.mark.parametrize("seed", [1, 2])
def test_kept_rows_move_together(d, nkv, page, seed):
    """Paths of any form (rows moved onto rows that move too), pages given back, sequences that end, keep all or nothing."""
    r = random.Random(seed)
    lens = [5, 16, 17, 40, 100, 130, 64, 200, 33]
    news = [5, 1, 17, 9, 70, 40, 64, 100, 0]
    kepts = [sorted(r.sample(range(T), r.randint(0, T))) for T in news]
    kepts[0], kepts[2], kepts[6], kepts[4] = list(range(5)), [], [0, 1, 63], list(range(0, 70, 2))
    order = r.sample(range(len(lens)), len(lens))
    pool = Pool(seed + d, lens, page, nkv, d)
    rows, news, kepts = order, [news[i] for i in order], [kepts[i] for i in order]
    assert _call(pool, rows, news, kepts) == [0] * len(lens)
    pool.keep_all(rows, news, kepts)
    pool.same()


def test_rows_by_their_number_and_many_sequences():
    r = random.Random(3)
    lens = [r.randint(1, 60) for _ in range(1500)]
    news = [r.randint(0, min(n, 9)) for n in lens]
    kepts = [sorted(r.sample(range(T), r.randint(0, T))) for T in news]
    pool = Pool(4, lens, 16, 1, 64, layers=1)
    assert _call(pool, None, news, kepts) == [0] * len(lens)
    pool.keep_all(range(1500), news, kepts)
    pool.same()


def test_refused_requests_change_nothing():
    """Bad lists, more drafts than tokens, sequences that are not there, shared pages; the others of the call are served."""
    lens, page = [40, 40, 40, 40, 30, 48, 48, 64, 40], 16
    news = [9, 9, 9, 50, 5, 16, 16, 32, 9]
    kepts = [[0, 5, 3], [0, 9], [-1, 2], [0, 1], [0, 2], [0, 2], list(range(16)), [], [0, 4]]
    # sequence 4's last page is shared, 5's too (it would hold kept drafts), 6's too (all stay), 7's too (only given back)
    pool = Pool(5, lens, page, 2, 64, shared=[(4, 1), (5, 2), (6, 2), (7, 3)])
    status = _call(pool, list(range(9)), news, kepts)
    assert status == [-1, -1, -1, -1, -1, -1, 0, 0, 0]
    pool.keep_all(range(9), news, kepts, refused=range(6))
    pool.same()
    assert qb.q_device_status() == qb.QB_OK


def test_sequences_and_counts_outside_their_range():
    pool = Pool(6, [20, 20], 16, 1, 64)
    status = _call(pool, [5, 1], [3, 3], [[0], [0, 2]])
    assert status == [-1, 0] and qb.q_device_status() == qb.QB_E_INDEX
    pool.keep_all([5, 1], [3, 3], [[0], [0, 2]], refused=[0])
    pool.same()
    for n in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        assert _call(pool, [0, 1], [3, 3], [[0], [0, 1, 2]], nkeep=[n, 3]) == [-1, 0]
        pool.same()
    assert _call(pool, [0, 1], [3, 3], None, keep=[2 ** 31 - 1] * 6, nkeep=[1, 1]) == [-1, -1]
    pool.same()


def test_a_bad_page_in_a_table_is_reported():
    pool = Pool(7, [40, 40], 16, 1, 64)
    pool.pages.tables[0, 2] = 1 << 20
    assert _call(pool, [0, 1], [9, 9], [[0, 5], [0, 3]]) == [-1, 0]
    assert qb.q_device_status() == qb.QB_E_INDEX and qb.q_device_status() == qb.QB_OK


def test_places_past_32_bits():
    """Two layers of more than 2^31 bytes each, the drafts on the last pages."""
    import torch
    nkv, d, page, npages = 8, 128, 64, 30000
    data = torch.empty((2, npages, nkv * qb.kv4_block_bytes(page, d)), dtype=torch.uint8, device="cuda")
    assert data.numel() > 2 ** 32
    table = [[npages - 1, npages - 3, npages - 2, -1]]
    pages = qb.KvPages(page, _i32([0]), _i32([-1] * npages), _i32([0] * (npages - 3) + [1] * 3), _i32([150]), _i32(table))
    slots = _i32([table[0][t // page] * page + t % page for t in range(150)])
    rows = torch.randn((2, 2, 150, nkv, d), generator=torch.Generator().manual_seed(1)).cuda()
    held, got = torch.empty_like(rows), torch.empty_like(rows)
    caches = [qb.Kv4(data[layer], page, nkv, d) for layer in (0, 1)]
    for cache, x, y in zip(caches, rows, held):
        qb.kv4_append(cache, x[0], x[1], slots)
        qb.kv4_read(cache, slots, y[0], y[1])
    kept, status = [1, 20, 59], _zeros(1)
    qb.kv4_keep(pages, data, nkv, d, None, _i32([0, 60]), _i32(kept + [-1] * 57), _i32([3]), status)
    for cache, y in zip(caches, got):
        qb.kv4_read(cache, slots, y[0], y[1])
    want = held.clone()
    want[:, :, 90:93] = held[:, :, [90 + k for k in kept]]
    assert status.tolist() == [0] and torch.equal(got, want)
    assert pages.lens.tolist() == [93] and pages.tables.tolist() == [[npages - 1, npages - 3, -1, -1]]
    assert int(pages.nfree) == 1 and int(pages.free[0]) == npages - 2


def test_nothing_to_do_and_refusals():
    import torch
    pool = Pool(8, [20], 16, 2, 64)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    qb.kv4_keep(pool.pages, pool.dev, 2, 64, e, _i32([0]), e, e, e)
    pool.same()
    one, start = _i32([1]), _i32([0, 1])
    for kw in (dict(nkv=1), dict(d=128), dict(q_start=one), dict(rows=_i32([0, 1])), dict(keep=one.float()), dict(status=e), dict(nkeep=one.cpu())):
        a = dict(nkv=2, d=64, rows=_i32([0]), q_start=start, keep=one, nkeep=one, status=one)
        a.update(kw)
        with pytest.raises(ValueError):
            qb.kv4_keep(pool.pages, pool.dev, a["nkv"], a["d"], a["rows"], a["q_start"], a["keep"], a["nkeep"], a["status"])
    for call in (lambda: qb.kv_tree_masks(one, one), lambda: qb.kv_tree_masks(one, _zeros(1, 1), _zeros(2)), lambda: qb.kv_tree_accept(one, _i32([1, 2]), one, one, one, one),
                 lambda: qb.kv_tree_accept(one, one, one, one, e, one)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(qb.QbError):
        qb.kv_tree_masks(one, _zeros(1, 33))
    qb.kv_tree_masks(e, torch.empty((0, 1), dtype=torch.int32, device="cuda"), q_start=_i32([0, 0]))
    pool.same()


def test_captured_and_replayed():
    """The whole round of a tree in one graph, on another state each time."""
    import torch
    r = random.Random(9)
    pools = [Pool(s, [60, 90], 16, 2, 128) for s in (1, 2, 3)]
    news = [12, 20]
    p = pools[0]
    parents, tokens, targets = (_zeros(32) for _ in range(3))
    masks, keep, nkeep, nxt, status = _zeros(32, 1), _zeros(32), _zeros(2), _zeros(2), _zeros(2)
    start, rows = _starts(news), _i32([1, 0])
    state = [p.pages.nfree, p.pages.free, p.pages.refs, p.pages.lens, p.pages.tables, p.dev]

    def round_():
        qb.kv_tree_masks(parents, masks, q_start=start)
        qb.kv_tree_accept(parents, tokens, targets, keep, nkeep, nxt, q_start=start)
        qb.kv4_keep(p.pages, p.dev, 2, 128, rows, start, keep, nkeep, status)

    parents.fill_(-1)
    saved = [t.clone() for t in state]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        round_()
    for s, q in enumerate(pools):
        for t, v in zip(state, saved if s == 0 else [q.pages.nfree, q.pages.free, q.pages.refs, q.pages.lens, q.pages.tables, q.dev]):
            t.copy_(v)
        trees = [tree(r, T, "tree") for T in news]
        toks = [[r.randrange(2) for _ in range(T)] for T in news]
        tgts = [[r.randrange(2) for _ in range(T)] for T in news]
        for t, v in zip((parents, tokens, targets), (trees, toks, tgts)):
            t.copy_(_i32(sum(v, [])))
        graph.replay()
        torch.cuda.synchronize()
        kepts = [walk(*x)[0] for x in zip(trees, toks, tgts)]
        assert nkeep.tolist() == [len(k) for k in kepts] and status.tolist() == [0, 0]
        q.keep_all([1, 0], news, kepts)
        q.pages, q.dev = p.pages, p.dev
        q.same()
