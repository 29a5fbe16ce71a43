"""The paged 4-bit cache on the GPU: stored bytes and values read back against
the plain definition bit for bit; attention against 64 bits.

Attention's tolerances.  A score is a sum of products whose magnitudes add up
to at most Z; each factor enters with a relative error of at most E (2^-21 with
f32 inputs, which enter as pairs of f16; 2^-11 with half-precision inputs, whose
products take one f16 factor) and the sums with at most A = 2^-19 of Z (f32
sums of up to a few hundred rounded terms a partial sum, and the rescalings).  So
a score is off by Z*(2E + A), a probability by twice that relatively (its own
exponent and the normalizing sum's), a product with a value by E + A more; the
output is rounded once.  A probability below 2^-38 may vanish (f16's least
number under a largest one of 2^14, as the header states): n keys with values of
at most V lose n*V*2^-38.
"""
import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
import kv4_ref as ref

pytestmark = pytest.mark.gpu

IN = {"f32": 2.0 ** -21, "f16": 2.0 ** -11, "bf16": 2.0 ** -11}
OUT = {"f32": 2.0 ** -23, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUM = 2.0 ** -19


def _type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qb.lib()
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


def _i32(a):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def _rows(rng, n, nkv, d, specials=False):
    x = (rng.standard_normal((n, nkv, d)) * np.float32(2.0) ** rng.integers(-3, 3, (n, nkv, 1))).astype(np.float32)
    if specials:
        x[0] = 0.0
        x[1, 0, 3] = np.inf
        x[2, 0, d - 1] = np.nan
        x[3] *= np.float32(1e-9)                    # steps that round to zero or to subnormals
        x[4] *= np.float32(1e6)                     # steps past binary16
        x[5] = np.float32(-2.5)                     # every element the extreme
        x[6, 0, :] = np.resize(np.float32([8, -8, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5]), d)  # extremes of both signs; ties
        x[7] = np.nan
    return x


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 64), (8, 16), (72, 64), (136, 16)])
def test_rows_bit_exact(name, d, page):
    """Stored bytes, values read back, slots passed over, strided inputs."""
    import torch
    rng = np.random.default_rng(d + page)
    nkv, n, npages = 3, 41, 7
    typ = _type(name)
    # keys and values lie in one wider buffer, as a fused projection leaves them
    wide = torch.from_numpy(np.concatenate([_rows(rng, n, nkv, d, True), _rows(rng, n, nkv, d, True)[::-1], _rows(rng, n, nkv, d)], 1)).cuda().to(typ)
    k, v = wide[:, :nkv], wide[:, nkv:2 * nkv]
    slots = rng.permutation(npages * page)[:n].astype(np.int32)
    slots[11] = -1
    pool = rng.integers(0, 256, (npages, nkv * ref.block_bytes(page, d)), dtype=np.uint8)
    got = torch.from_numpy(pool).cuda()
    cache = qb.Kv4(got, page, nkv, d)
    qb.kv4_append(cache, k, v, _i32(slots))
    kn, vn = k.float().cpu().numpy(), v.float().cpu().numpy()
    for i in range(n):
        if slots[i] >= 0:
            ref.write_row(pool, page, nkv, d, slots[i], kn[i], vn[i])
    assert np.array_equal(got.cpu().numpy(), pool)
    for out in ("f32", name):
        kb, vb = (torch.full((n, nkv, d), 7.0, dtype=_type(out), device="cuda") for _ in "kv")
        qb.kv4_read(cache, _i32(slots), kb, vb)
        for i in range(n):
            wk, wv = ref.read_row(pool, page, nkv, d, slots[i]) if slots[i] >= 0 else (np.zeros((nkv, d)),) * 2
            for g, w in ((kb, wk), (vb, wv)):
                want = torch.from_numpy(w.astype(np.float32)).to(_type(out))
                assert torch.equal(torch.nan_to_num(g[i].cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))


def test_rows_slot_past_the_cache_is_reported():
    import torch
    data = torch.zeros((4, qb.kv4_block_bytes(16, 64)), dtype=torch.uint8, device="cuda")
    x = torch.ones((2, 1, 64), device="cuda")
    qb.kv4_append(qb.Kv4(data, 16, 1, 64), x, x, _i32([64, 5]))
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert qb.q_device_status() == qb.QB_OK
    a, b = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
    qb.kv4_read(qb.Kv4(data, 16, 1, 64), _i32([1 << 20, 5]), a, b)
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert a[0].abs().max() == 0 and torch.equal(a[1], x[1]) and torch.equal(b[1], x[1])


class Batch:
    """Sequences of given lengths in a pool whose other bytes are all ones (NaN steps)."""

    def __init__(self, seed, lens, news, nh, nkv, d, page, name, spare=3, offset=0.5, kmul=1.0):
        import torch
        rng = np.random.default_rng(seed)
        self.lens, self.news, self.nh, self.nkv, self.d, self.page, self.name = lens, news, nh, nkv, d, page, name
        need = [-(-n // page) for n in lens]
        npages = sum(need) + spare
        ids = rng.permutation(npages)
        maxp = max(max(need), 1) + 1
        self.tables = np.full((len(lens), maxp), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.pool = torch.full((npages, nkv * ref.block_bytes(page, d)), 255, dtype=torch.uint8, device="cuda")
        self.cache = qb.Kv4(self.pool, page, nkv, d)
        shift = rng.standard_normal((1, nkv, d)) * offset
        total = sum(lens)
        k = torch.from_numpy(((rng.standard_normal((total, nkv, d)) + shift) * kmul).astype(np.float32)).cuda()
        v = torch.from_numpy(rng.standard_normal((total, nkv, d)).astype(np.float32)).cuda()
        slots = np.concatenate([self.tables[s, np.arange(n) // page] * page + np.arange(n) % page for s, n in enumerate(lens)] + [np.zeros(0, np.int32)])
        if total:
            qb.kv4_append(self.cache, k, v, _i32(slots))
            kb, vb = torch.empty_like(k), torch.empty_like(v)
            qb.kv4_read(self.cache, _i32(slots), kb, vb)
            self.k, self.v = kb.double().cpu().numpy(), vb.double().cpu().numpy()
        else:
            self.k = self.v = np.zeros((0, nkv, d))
        self.q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.q = torch.from_numpy(rng.standard_normal((sum(news), nh, d)).astype(np.float32)).cuda().to(_type(name))

    def run(self, scale, window=0, rows=None, stream=None, q_start=True):
        import torch
        seqs = qb.KvSeqs(_i32(self.tables), _i32(self.lens), rows=rows, q_start=_i32(self.q_start) if q_start else None)
        out = torch.full_like(self.q, 9.0)
        lse = torch.full(self.q.shape[:2], 9.0, device="cuda")
        qb.kv4_attn(self.cache, self.q, seqs, scale, out, lse=lse, window=window)
        torch.cuda.synchronize()
        return out, lse

    def want(self, scale, window=0):
        parts, at = [], 0
        q = self.q.double().cpu().numpy()
        for s, (n, T) in enumerate(zip(self.lens, self.news)):
            a = self.q_start[s]
            parts.append(ref.attention(q[a:a + T], self.k[at:at + n], self.v[at:at + n], n, T, scale, window))
            at += n
        return [np.concatenate(x) for x in zip(*parts)]

    def check(self, scale=None, window=0, **kw):
        scale = self.d ** -0.5 if scale is None else scale
        out, lse = self.run(scale, window, **kw)
        want, wlse, zabs, mag = self.want(scale, window)
        e = IN[self.name]
        off = zabs * (2 * e + SUM)
        tol = (2 * off + e + SUM)[..., None] * mag + OUT[self.name] * np.abs(want) + 2.0 ** -24 * (self.name != "f32")
        tol += len(self.v) * np.abs(self.v).max(initial=0) * 2.0 ** -38
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / np.maximum(tol, 1e-30))
        gl = lse.double().cpu().numpy()
        empty = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(gl), empty)
        lt = off + SUM * (1 + np.abs(np.where(empty, 0, wlse)))
        assert np.all(np.abs(gl[~empty] - wlse[~empty]) <= lt[~empty])
        assert np.all(got[empty] == 0)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nh,nkv,d,page", [(4, 1, 128, 16), (9, 3, 64, 32), (8, 1, 256, 64), (5, 1, 80, 16), (16, 1, 128, 64), (17, 1, 64, 16),
                                           (2, 2, 256, 16), (3, 3, 8, 32)])
def test_single_tokens(name, nh, nkv, d, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 64, 65, 0, 100, 257, 300]
    Batch(nh + d, lens, [1] * len(lens), nh, nkv, d, page, name).check(q_start=False)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("window", [0, 1, 7, 40])
@pytest.mark.parametrize("nh,nkv,d,page", [(8, 2, 128, 16), (9, 3, 64, 64), (4, 2, 256, 32)])
def test_several_tokens(name, window, nh, nkv, d, page):
    """Drafted tokens and short prompts: ragged, some longer than their cache (rows that see nothing), some without tokens."""
    Batch(nh + window, [40, 3, 70, 0, 130, 64, 1], [5, 8, 70, 2, 33, 0, 1], nh, nkv, d, page, name).check(window=window)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nh,nkv,d,page", [(4, 1, 128, 64), (3, 1, 64, 16), (2, 1, 256, 32), (8, 2, 96, 16)])
def test_prompts(name, nh, nkv, d, page):
    Batch(nh, [333, 200, 129], [333, 61, 128], nh, nkv, d, page, name).check()


@pytest.mark.parametrize("name", ["f32", "bf16"])
def test_prompt_window(name):
    Batch(3, [300, 170], [260, 170], 4, 2, 128, 16, name).check(window=50)


@pytest.mark.parametrize("name", ["f32", "f16"])
def test_long_sequences_are_split(name):
    Batch(5, [9001, 40, 5000], [1, 1, 2], 4, 1, 128, 16, name).check()


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_sharp_and_large_scores(name):
    """Scores of hundreds: the running maximum moves, most probabilities vanish."""
    Batch(7, [700, 90], [1, 3], 4, 2, 64, 16, name, kmul=12.0).check(scale=1.0)


def test_small_and_large_values():
    """Steps from binary16's subnormals to its top in one sequence: the values' scale moves along the keys."""
    import torch
    b = Batch(8, [200], [2], 4, 1, 128, 16, "f32")
    v = np.random.default_rng(1).standard_normal((200, 1, 128)) * 10.0 ** np.linspace(-5, 4.5, 200)[:, None, None]
    slots = _i32(b.tables[0, np.arange(200) // 16] * 16 + np.arange(200) % 16)
    k = torch.from_numpy(b.k.astype(np.float32)).cuda()
    vt = torch.from_numpy(v.astype(np.float32)).cuda()
    qb.kv4_append(b.cache, k, vt, slots)
    kb, vb = torch.empty_like(k), torch.empty_like(vt)
    qb.kv4_read(b.cache, slots, kb, vb)
    b.k, b.v = kb.double().cpu().numpy(), vb.double().cpu().numpy()
    b.check()


def test_unreadable_rows_reach_their_own_heads_only():
    """An infinity in a key or a value makes the outputs that see it NaN, and no others."""
    import torch
    b = Batch(9, [90, 90, 90], [1, 1, 1], 4, 2, 64, 16, "f32")
    clean, _ = b.run(0.125)
    x = torch.from_numpy(np.stack([b.k, b.v]).astype(np.float32)).cuda()
    x[0, 90 + 17, 1, 5] = float("inf")    # sequence 1, key 17, key head 1
    x[1, 180 + 88, 0, 40] = -float("inf")  # sequence 2, value 88, key head 0
    slots = _i32(np.concatenate([b.tables[s, np.arange(90) // 16] * 16 + np.arange(90) % 16 for s in range(3)]))
    qb.kv4_append(b.cache, x[0].contiguous(), x[1].contiguous(), slots)
    out, lse = b.run(0.125)
    assert torch.equal(out[0], clean[0])
    assert out[1, 2:].isnan().all() and lse[1, 2:].isnan().all() and torch.equal(out[1, :2], clean[1, :2])
    assert out[2, :2, 32:].isnan().all() and not out[2, 2:].isnan().any() and torch.equal(out[2, 2:], clean[2, 2:])


def test_rows_choose_and_share_tables():
    import torch
    b = Batch(11, [50, 20, 33], [1, 1, 1], 4, 2, 64, 16, "f32")
    out, _ = b.run(0.125)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens), rows=_i32([2, 0, 2, 1]))
    q = b.q[[2, 0, 2, 1]].contiguous()
    got = torch.empty_like(q)
    qb.kv4_attn(b.cache, q, seqs, 0.125, got)
    assert torch.equal(got, out[[2, 0, 2, 1]])


def test_strided_queries_and_outputs():
    import torch
    b = Batch(12, [70, 5], [1, 1], 4, 2, 64, 16, "bf16")
    want, _ = b.run(0.125)
    wide_q = torch.zeros((2, 9, 64), dtype=torch.bfloat16, device="cuda")
    wide_o = torch.full((2, 6, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    wide_q[:, 2:6] = b.q
    qb.kv4_attn(b.cache, wide_q[:, 2:6], qb.KvSeqs(_i32(b.tables), _i32(b.lens)), 0.125, wide_o[:, 1:5])
    assert torch.equal(wide_o[:, 1:5], want) and (wide_o[:, 0] == 3).all() and (wide_o[:, 5] == 3).all()


def test_same_bits_twice_and_on_another_stream():
    import torch
    b = Batch(13, [3000, 1, 700], [1, 1, 1], 8, 2, 128, 16, "f32")
    one, l1 = b.run(0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        two, l2 = b.run(0.1)
    assert torch.equal(one, two) and torch.equal(l1, l2)


def test_captured_in_a_graph():
    import torch
    b = Batch(14, [500, 40], [1, 1], 8, 2, 128, 16, "bf16")
    want, _ = b.run(0.1)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens))
    out = torch.zeros_like(b.q)
    ws = torch.empty(qb.kv4_attn_workspace_bytes(b.cache, b.q), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            qb.kv4_attn(b.cache, b.q, seqs, 0.1, out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A cache of over 4 GiB whose last pages hold the sequence."""
    import torch
    page, nkv, d = 64, 8, 256
    per = nkv * ref.block_bytes(page, d)
    npages = (1 << 32) // per + 40
    pool = torch.zeros((npages, per), dtype=torch.uint8, device="cuda")
    cache = qb.Kv4(pool, page, nkv, d)
    rng = np.random.default_rng(15)
    n = 130
    k = torch.from_numpy(rng.standard_normal((n, nkv, d)).astype(np.float32)).cuda()
    v = torch.from_numpy(rng.standard_normal((n, nkv, d)).astype(np.float32)).cuda()
    tables = np.array([[npages - 1, npages - 17, npages - 30]], np.int32)
    slots = _i32(tables[0, np.arange(n) // page].astype(np.int64) * page + np.arange(n) % page)
    qb.kv4_append(cache, k, v, slots)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    qb.kv4_read(cache, slots, kb, vb)
    assert (kb - k).abs().max() < 1.0 and (vb - v).abs().max() < 1.0
    q = torch.from_numpy(rng.standard_normal((1, 16, d)).astype(np.float32)).cuda()
    out = torch.empty_like(q)
    qb.kv4_attn(cache, q, qb.KvSeqs(_i32(tables), _i32([n])), 0.0625, out)
    want = ref.attention(q.double().cpu().numpy(), kb.double().cpu().numpy(), vb.double().cpu().numpy(), n, 1, 0.0625, 0)
    off = want[2] * (2 * IN["f32"] + SUM)
    tol = (2 * off + IN["f32"] + SUM)[..., None] * want[3] + OUT["f32"] * np.abs(want[0])
    assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= tol)


def test_indices_outside_the_cache_are_reported():
    import torch
    b = Batch(16, [40, 20], [1, 1], 2, 1, 64, 16, "f32")
    want, _ = b.run(0.125)
    b.tables[1, 0] = 1 << 20
    out, _ = b.run(0.125)
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert torch.equal(out[0], want[0])
    b.tables[1, 0] = 0
    out, lse = b.run(0.125, rows=_i32([0, 7]))
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert torch.equal(out[0], want[0]) and (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_a_length_past_its_table_row_is_cut():
    import torch
    b = Batch(17, [48], [1], 2, 1, 64, 16, "f32")
    b.tables = b.tables[:, :3].copy()
    want, _ = b.run(0.125)
    b.lens = [5000]
    got, _ = b.run(0.125)
    assert torch.equal(got, want)


# ---------------------------------------------------------------- pages

class State:
    def __init__(self, page, npages, nrows, maxp, layers, words):
        import torch
        self.d = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in
                  (("nfree", (1,)), ("free", (npages,)), ("refs", (npages,)), ("lens", (nrows,)), ("tables", (nrows, maxp)))}
        self.h = qb.KvPages(page, *(self.d[n] for n in ("nfree", "free", "refs", "lens", "tables")))
        pool = np.random.default_rng(0).integers(0, 1 << 30, (layers, npages, words), dtype=np.int32)
        self.pool = torch.from_numpy(pool).cuda()
        self.ref = ref.Pages(page, npages, nrows, maxp, pool=pool.copy())
        qb.kv_pages_reset(self.h)

    def same(self):
        r, d = self.ref, {k: v.cpu().numpy() for k, v in self.d.items()}
        assert d["nfree"][0] == len(r.stack)
        assert d["free"][:len(r.stack)].tolist() == r.stack
        assert d["refs"].tolist() == r.refs
        assert d["lens"].tolist() == r.lens
        assert d["tables"].tolist() == [row + [-1] * (r.maxp - len(row)) for row in r.rows]
        assert np.array_equal(self.pool.cpu().numpy(), r.pool)


@pytest.mark.parametrize("page,npages,nrows,maxp,layers,words,seed", [(16, 26, 12, 9, 2, 36, 0), (64, 33, 40, 4, 1, 1028, 1), (32, 1500, 1100, 6, 3, 4, 2)])
def test_pages_follow_the_model(page, npages, nrows, maxp, layers, words, seed):
    """A random run of extend, fork, free, compact: the whole state and every byte after each call, requests that do not fit among them."""
    import torch
    st = State(page, npages, nrows, maxp, layers, words)
    st.same()
    rng = np.random.default_rng(seed)
    refused = 0
    for step in range(30):
        op = rng.choice(["extend", "extend", "fork", "free", "compact"])
        if op == "extend":
            n = int(rng.integers(1, nrows + 1))
            rows = rng.permutation(nrows)[:n]
            counts = rng.integers(0, 2 * page, n)
            want, wst = st.ref.extend(rows.tolist(), counts.tolist())
            slots = torch.full((len(want) + 1,), -7, dtype=torch.int32, device="cuda")
            status = torch.full((n,), 5, dtype=torch.int32, device="cuda")
            qb.kv_pages_extend(st.h, _i32(rows), _i32(counts), slots, status)
            assert slots.tolist() == want + [-7] and status.tolist() == wst
            refused += sum(s == -8 for s in wst)
        elif op == "fork":
            empty = [r for r in range(nrows) if not st.ref.lens[r]]
            full = [r for r in range(nrows) if st.ref.lens[r]]
            if not empty or not full:
                continue
            n = int(rng.integers(1, len(empty) + 1))
            children = rng.permutation(empty)[:n].tolist()
            parents = rng.choice(full, n).tolist()
            want = st.ref.fork(parents, children)
            status = torch.full((n,), 5, dtype=torch.int32, device="cuda")
            qb.kv_pages_fork(st.h, st.pool, _i32(parents), _i32(children), status)
            assert status.tolist() == want
            refused += sum(s == -8 for s in want)
        elif op == "free":
            rows = rng.permutation(nrows)[:int(rng.integers(1, nrows + 1))].tolist()
            st.ref.free(rows)
            qb.kv_pages_free(st.h, _i32(rows))
        else:
            st.ref.compact()
            qb.kv_pages_compact(st.h, st.pool)
        st.same()
    assert refused > 0
    assert qb.q_device_status() == qb.QB_OK


def test_pages_refusals_on_the_device():
    import torch
    st = State(16, 6, 4, 2, 1, 4)
    status = torch.empty(3, dtype=torch.int32, device="cuda")
    slots = torch.full((50,), -7, dtype=torch.int32, device="cuda")
    # an outside sequence, a negative count, a request past its table row
    qb.kv_pages_extend(st.h, _i32([9, 1, 2]), _i32([3, -1, 33]), slots, status)
    assert status.tolist() == [qb.QB_E_ARG, qb.QB_E_ARG, qb.QB_E_PAGES]
    assert slots.tolist() == [-1] * 36 + [-7] * 14
    assert qb.q_device_status() == qb.QB_E_INDEX
    st.same()
    st.ref.extend([0, 1], [20, 16])
    qb.kv_pages_extend(st.h, _i32([0, 1]), _i32([20, 16]), slots, status)
    # a child that is not empty
    qb.kv_pages_fork(st.h, st.pool, _i32([0, 0]), _i32([1, 3]), status)
    assert status.tolist()[:2] == [qb.QB_E_ARG, 0]
    st.ref.fork([0, 0], [1, 3])
    st.same()
    # an outside sequence is passed over by free
    st.ref.free([0, 3])
    qb.kv_pages_free(st.h, _i32([0, 77, 3]))
    assert qb.q_device_status() == qb.QB_E_INDEX
    st.same()


def test_pages_copy():
    import torch
    pool = torch.randint(0, 1 << 30, (3, 20, 260), dtype=torch.int32, device="cuda")
    want = pool.clone()
    want[:, [7, 0, 19]] = want[:, [3, 12, 5]]
    qb.kv_pages_copy(pool, 20, _i32([3, 12, 5]), _i32([7, 0, 19]))
    assert torch.equal(pool, want)
    qb.kv_pages_copy(pool, 20, _i32([3, 20]), _i32([4, 2]))
    want[:, 4] = want[:, 3]
    assert qb.q_device_status() == qb.QB_E_INDEX
    assert torch.equal(pool, want)


def test_a_serving_loop():
    """Pages, rows and attention together: prompts, a fork, single tokens; the attention equals one over the same rows laid out by hand."""
    import torch
    rng = np.random.default_rng(21)
    page, nkv, nh, d, npages = 16, 2, 4, 64, 40
    st = State(page, npages, 5, 8, 1, nkv * ref.block_bytes(page, d) // 4)
    cache = qb.Kv4(st.pool[0].view(torch.uint8), page, nkv, d)
    held = {r: [] for r in range(5)}

    def grow(rows, counts):
        total = sum(counts)
        slots = torch.empty(total, dtype=torch.int32, device="cuda")
        status = torch.empty(len(rows), dtype=torch.int32, device="cuda")
        qb.kv_pages_extend(st.h, _i32(rows), _i32(counts), slots, status)
        k, v, q = (torch.from_numpy(rng.standard_normal((total, h, d)).astype(np.float32)).cuda() for h in (nkv, nkv, nh))
        qb.kv4_append(cache, k, v, slots)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        qb.kv4_read(cache, slots, kb, vb)
        start = np.concatenate([[0], np.cumsum(counts)])
        out = torch.empty_like(q)
        qb.kv4_attn(cache, q, qb.KvSeqs(st.d["tables"], st.d["lens"], rows=_i32(rows), q_start=_i32(start)), 0.125, out)
        for i, r in enumerate(rows):
            held[r] += list(zip(kb[start[i]:start[i + 1]].double().cpu().numpy(), vb[start[i]:start[i + 1]].double().cpu().numpy()))
            kk, vv = (np.stack([x[j] for x in held[r]]) for j in (0, 1))
            want, _, zabs, mag = ref.attention(q[start[i]:start[i + 1]].double().cpu().numpy(), kk, vv, len(kk), counts[i], 0.125, 0)
            off = zabs * (2 * IN["f32"] + SUM)
            tol = (2 * off + IN["f32"] + SUM)[..., None] * mag + OUT["f32"] * np.abs(want)
            assert np.all(np.abs(out[start[i]:start[i + 1]].double().cpu().numpy() - want) <= tol)

    grow([0, 2], [37, 20])
    status = torch.empty(2, dtype=torch.int32, device="cuda")
    qb.kv_pages_fork(st.h, st.pool, _i32([0, 2]), _i32([1, 4]), status)
    held[1], held[4] = list(held[0]), list(held[2])
    for _ in range(3):
        grow([4, 0, 1, 2], [1, 1, 1, 1])
    qb.kv_pages_free(st.h, _i32([0]))
    held[0] = []
    qb.kv_pages_compact(st.h, st.pool)
    grow([1, 0, 4], [2, 18, 1])


# ---------------------------------------------------------------- prompts out of the ordinary

def _fill(b, k, v):
    """Writes rows k, v [n, nkv, d] over a one-sequence batch's cache and takes what they read back as."""
    import torch
    n = b.lens[0]
    slots = _i32(b.tables[0, np.arange(n) // b.page] * b.page + np.arange(n) % b.page)
    kt, vt = (torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda() for x in (k, v))
    qb.kv4_append(b.cache, kt, vt, slots)
    kb, vb = torch.empty_like(kt), torch.empty_like(vt)
    qb.kv4_read(b.cache, slots, kb, vb)
    b.k, b.v = kb.double().cpu().numpy(), vb.double().cpu().numpy()


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_large_steps(name, d):
    """Steps past 2^12 in single keys, values and groups, small ones beside them."""
    b = Batch(31, [300], [200], 4, 2, d, 16, name)
    k, v = b.k.copy(), b.v.copy()
    v[40:44, 0] *= 8e4
    v[150, 1, 32:40] = 3e5
    k[77, 1] *= 6e4 * np.sign(np.arange(d) - 9.5)
    b.q *= 0.001
    _fill(b, k, v)
    assert np.isfinite(b.k).all() and np.isfinite(b.v).all()
    b.check()


@pytest.mark.parametrize("name", ["f32", "f16"])
@pytest.mark.parametrize("nh,nkv,d,T", [(4, 2, 64, 200), (2, 1, 128, 170), (2, 1, 128, 3)])
def test_unreadable_rows_in_prompts(name, nh, nkv, d, T):
    """An infinite value makes its group's outputs NaN in the rows that see it, an infinite key every output; rows before them and other heads stay."""
    import torch
    n = 260
    b = Batch(32, [n], [T], nh, nkv, d, 32, name)
    clean, clean_lse = b.run(0.125)
    k, v = b.k.copy(), b.v.copy()
    kv, kk = n - T // 2 - 1, n - T // 4 - 1     # places of the bad value and of the bad key
    v[kv, 0, d - 1] = np.inf
    k[kk, nkv - 1, 5] = -np.inf
    _fill(b, k, v)
    out, lse = b.run(0.125)
    grp = nh // nkv
    pos = n - T + np.arange(T)
    for h in range(nh):
        saw_v = (pos >= kv) & (h // grp == 0)
        saw_k = (pos >= kk) & (h // grp == nkv - 1)
        o, c = out[:, h].float().cpu().numpy(), clean[:, h].float().cpu().numpy()
        same = ~(saw_v | saw_k)
        assert np.array_equal(o[same], c[same])
        assert np.isnan(o[saw_k]).all() and lse[:, h].isnan().cpu().numpy()[saw_k].all()
        only_v = saw_v & ~saw_k
        last = np.arange(d) >= (d - 1) // 32 * 32
        assert np.isnan(o[only_v][:, last]).all() and not np.isnan(o[only_v][:, ~last]).any()
        assert torch.equal(lse[:, h][torch.from_numpy(only_v).cuda()], clean_lse[:, h][torch.from_numpy(only_v).cuda()])


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 3e-6])
@pytest.mark.parametrize("T", [1, 150])
def test_scales(name, scale, T):
    """Negative, zero and small factors: the largest score is the one after the factor."""
    Batch(33, [190], [T], 4, 2, 64, 64, name).check(scale=scale)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_prompt_sharp_scores(name):
    """Scores that rise by hundreds along the keys: the maximum moves within and between tiles."""
    b = Batch(34, [520], [400], 4, 2, 128, 16, name, offset=0.0)
    ramp = np.linspace(0.0, 30.0, 520)[:, None, None]
    _fill(b, b.k * 0.1 + ramp, b.v)
    b.q.abs_()
    b.check()


@pytest.mark.parametrize("name", ["f32", "f16"])
def test_prompts_of_many_sequences(name):
    """More than a table's 64 sequences, some empty, some without new tokens, tables chosen by rows."""
    import torch
    rng = np.random.default_rng(35)
    lens = [int(x) for x in rng.integers(0, 150, 90)]
    news = [int(rng.integers(0, 80)) if i % 7 else 0 for i in range(90)]
    b = Batch(35, lens, news, 4, 2, 64, 16, name)
    b.check()
    perm = rng.permutation(90)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(lens), rows=_i32(perm), q_start=_i32(np.concatenate([[0], np.cumsum(np.array(news)[perm])])))
    out, _ = b.run(0.125)
    pick = np.concatenate([np.arange(b.q_start[s], b.q_start[s + 1]) for s in perm]).astype(np.int64)
    q = b.q[torch.from_numpy(pick).cuda()].contiguous()
    got = torch.empty_like(q)
    qb.kv4_attn(b.cache, q, seqs, 0.125, got)
    want = out[torch.from_numpy(pick).cuda()]
    # which keys a warp holds depends on the order: the same up to the sums' rounding
    tol = 2.0 ** -17 if name == "f32" else 2.0 ** -9
    assert (got.float() - want.float()).abs().max() <= tol * max(1.0, float(want.float().abs().max()))


def test_prompt_same_bits_twice():
    import torch
    b = Batch(36, [700, 300], [400, 300], 8, 2, 128, 16, "bf16")
    one, l1 = b.run(0.1)
    two, l2 = b.run(0.1)
    assert torch.equal(one, two) and torch.equal(l1, l2)


def test_prompt_strided_and_window_and_page_32():
    import torch
    b = Batch(37, [400], [300], 4, 2, 64, 32, "f16")
    want, _ = b.run(0.125, window=130)
    wide_q = torch.zeros((300, 8, 64), dtype=torch.float16, device="cuda")
    wide_o = torch.full((300, 6, 64), 3.0, dtype=torch.float16, device="cuda")
    wide_q[:, 4:] = b.q
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens), q_start=_i32(b.q_start))
    qb.kv4_attn(b.cache, wide_q[:, 4:], seqs, 0.125, wide_o[:, 1:5], window=130)
    assert torch.equal(wide_o[:, 1:5], want) and (wide_o[:, 0] == 3).all() and (wide_o[:, 5] == 3).all()
    b.check(window=130)
