"""The paged 4-bit cache at its edges on the GPU."""
import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
import kv4_ref as ref
from test_gpu_kv4 import OUT, SUM, Batch, _fill, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qb.lib()
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


@pytest.mark.parametrize("call", ["copy", "fork", "compact"])
def test_scores_right_after_page_copies(call):
    """Pages of the int8 key cache are copied and scored at once: the scores are those of the copied rows."""
    import torch
    nkv, nh, d, page, half = 4, 8, 128, 16, 1024
    npages = 2 * half
    lcap = npages * page
    rng = np.random.default_rng(61)
    qc = torch.from_numpy(rng.integers(-127, 128, (nh, d), dtype=np.int8)).cuda()
    qs = torch.full((nh, 1), 128, dtype=torch.int32, device="cuda")           # 128 * 2^0
    ks = torch.full((nkv, lcap), 0x3C00, dtype=torch.int16, device="cuda")    # 1.0
    for turn in range(4):
        kc = torch.from_numpy(rng.integers(-127, 128, (nkv, lcap, d), dtype=np.int8)).cuda()
        want_kc = kc.clone().view(nkv, npages, page * d)
        want_kc[:, :half] = want_kc[:, half:]                                  # page half + i to page i
        want, got = (torch.zeros((nh, lcap), device="cuda") for _ in range(2))
        qb.kv_scores(qb.PERBLOCK, qc, qs, d, want_kc.view(nkv, lcap, d), ks, lcap, 0.125, want)
        data = kc.view(nkv, npages, page * d)
        refs = np.zeros(npages, np.int32)
        refs[half:] = 1
        free = np.concatenate([np.arange(half)[::-1], np.full(half, -1)])      # page 0 the next to go
        status = torch.zeros(half, dtype=torch.int32, device="cuda")
        if call == "compact":                                                  # one sequence holds the upper half
            tables, lens = np.arange(half, npages)[None], [half * page]
        else:                                                                  # each page a sequence of its own, partly filled
            tables = np.full((npages, 1), -1)
            tables[:half, 0] = np.arange(half, npages)
            lens = [page - 1] * half + [0] * half
        pages = qb.KvPages(page, _i32([half]), _i32(free), _i32(refs), _i32(lens), _i32(tables))
        work = torch.empty(qb.kv_pages_workspace_bytes(pages), dtype=torch.uint8, device="cuda")
        lo, hi = _i32(np.arange(half)), _i32(np.arange(half, npages))
        torch.cuda.synchronize()
        if call == "copy":
            qb.kv_pages_copy(data, npages, hi, lo)
        elif call == "fork":
            qb.kv_pages_fork(pages, data, lo, hi, status, work)
        else:
            qb.kv_pages_compact(pages, data, work)
        qb.kv_scores(qb.PERBLOCK, qc, qs, d, kc, ks, lcap, 0.125, got)
        assert torch.equal(got, want) and int(status.min()) == 0
        assert torch.equal(kc, want_kc.view(nkv, lcap, d))


def test_slots_of_requests_of_any_count():
    """Refused requests of up to 2^31 - 1 tokens, and an array of slots that ends in the middle: nothing outside is written."""
    import torch
    page, npages, nrows, maxp = 16, 40, 8, 4
    d = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, npages, npages, nrows, (nrows, maxp))]
    pages = qb.KvPages(page, *d)
    for counts, nslots, want_status in (([3, 2 ** 31 - 1, 5], 50, [0, -8, 0]), ([2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 20], 7, [-8] * 3),
                                        ([20, 1 << 30, 4], 22, [0, -8, 0]), ([64, 2 ** 31 - 31, 64], 0, [0, -8, 0])):
        qb.kv_pages_reset(pages)
        wide = torch.full((nslots + 4096,), -7, dtype=torch.int32, device="cuda")
        slots = wide[2048:2048 + nslots] if nslots else wide[2048:2048]
        status = torch.full((3,), 5, dtype=torch.int32, device="cuda")
        rows = [1, 2, 3]
        if nslots:
            qb.kv_pages_extend(pages, _i32(rows), _i32(counts), slots, status)
        else:  # the entry itself: an array of no entries
            from block_quantized_weight_quantize_gb300 import kv4
            r, c = _i32(rows), _i32(counts)
            assert kv4._c.kv_pages_extend(pages.ref, r.data_ptr(), c.data_ptr(), 3, wide.data_ptr() + 8192, 0, status.data_ptr(),
                                          torch.cuda.current_stream().cuda_stream) == qb.QB_OK
        assert status.tolist() == want_status
        want, page_at = [], 0
        for n, st in zip(counts, want_status):
            want += [page * page_at + t if st == 0 else -1 for t in range(min(n, 64))] if st == 0 else [-1] * min(n, nslots)
            page_at += -(-n // page) if st == 0 else 0
        assert slots.tolist() == want[:nslots]
        assert (wide[:2048] == -7).all() and (wide[2048 + nslots:] == -7).all()
        assert d[3].tolist()[1:4] == [n if st == 0 else 0 for n, st in zip(counts, want_status)]
        assert qb.q_device_status() == qb.QB_E_INDEX


# A row's probabilities next to a key far above the others.  Tolerance, from the stored values: a score is off by at most
# its magnitudes' sum Z times 2^-19 (f32 sums; queries are exact in f16, keys as two f16) or times 2^-11 more where keys are
# rounded to f16 (a row that sees 2048 keys or more), a probability by twice that relatively, probabilities and values are f16 (2^-11 each, or
# one product of 2^-11 in the step kernel), the output is rounded once, and each probability may lose `low` of the largest (as the header states).
# An f16 output has an absolute 2^-25 besides (its least place).

def _check_probabilities(b, name, scale, low, dims=slice(None)):
    out, lse = b.run(scale)
    want, wlse, zabs, mag = b.want(scale)
    off = zabs * (SUM + (2.0 ** -11 if b.lens[0] - b.news[0] + 1 >= 2048 else 0.0))
    tol = (2 * off + 2.0 ** -10 + SUM)[..., None] * mag + OUT[name] * np.abs(want) + 2.0 ** -25 * (name == "f16")
    tol += len(b.v) * np.abs(b.v).max() * low
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got - want)[..., dims] <= tol[..., dims]), np.max((np.abs(got - want) / tol)[..., dims])
    assert np.all(np.abs(lse.double().cpu().numpy() - wlse) <= off + SUM * (1 + np.abs(wlse)))


def _beside_one_key(name, d, n, T, gap, place, seed=71):
    """Queries u + noise; key `place` is gap nats above the others for every row, its value zero, the others' 30 +- 10."""
    b = Batch(seed, [n], [T], 2, 1, d, 32, name)
    rng = np.random.default_rng(seed)
    u = np.where(np.arange(d) % 2, 1.0, -1.0)
    import torch
    b.q = torch.from_numpy((u + 0.05 * rng.standard_normal((T, 2, d))).astype(np.float32)).cuda().to(b.q.dtype)
    k = rng.standard_normal((n, 1, d)) * 0.05
    v = 30.0 + 10.0 * rng.standard_normal((n, 1, d))
    k[place, 0] = u * gap * d ** -0.5
    v[place] = 0.0
    _fill(b, k, v)
    return b


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("gap", [10.0, 18.0, 21.0])
@pytest.mark.parametrize("d,n,T,place", [(64, 1900, 100, 3), (128, 900, 100, 780), (128, 2300, 120, 0), (64, 300, 20, 3), (64, 900, 100, 110),
                                             (128, 700, 300, 95)])
def test_small_probabilities_beside_a_large_one(name, gap, d, n, T, place):
    """Probabilities of 2^-14 to 2^-30 of the largest make up the output, through both kernels; the large one comes first, or late in a
    tile of 128 keys."""
    _check_probabilities(_beside_one_key(name, d, n, T, gap, place), name, d ** -0.5, 2.0 ** (-36 if T >= 100 else -38))


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("at", [5, 130, 640])
def test_small_probabilities_beside_a_large_value(name, at):
    """The same with a value of steps past 2^12 in one group of a key without weight in the sum: the other groups' outputs."""
    d = 128
    b = _beside_one_key(name, d, 700, 100, 12.0, 3)
    v = b.v.copy()
    v[at, 0, 32:64] = np.resize([3e5, -3e5], 32)
    k = b.k.copy()
    u = np.where(np.arange(d) % 2, 1.0, -1.0)
    k[at, 0] = -u * 40.0 * d ** -0.5
    _fill(b, k, v)
    big = b.v[:, :, 32:64].copy()
    b.v[at, 0, 32:64] = 0.0     # the sum of magnitudes in the bound is that of the other groups
    try:
        _check_probabilities(b, name, d ** -0.5, 2.0 ** -32, np.r_[0:32, 64:128])
    finally:
        b.v[:, :, 32:64] = big


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nh,nkv,d,page,T,window", [(1, 1, 64, 16, 3, 0), (4, 2, 128, 64, 5, 0), (8, 1, 256, 32, 3, 0), (4, 1, 128, 16, 1, 50), (12, 2, 64, 64, 1, 50),
                                                    (3, 1, 256, 16, 1, 50), (4, 2, 64, 16, 150, 0), (4, 1, 128, 32, 70, 45)])
def test_finite_keys_and_values_that_a_token_does_not_see(name, nh, nkv, d, page, T, window):
    """A key and a value near the top of the format's range in one place: tokens that do not see it keep their bits."""
    import torch
    n = 190
    b = Batch(81, [n], [T], nh, nkv, d, page, name)
    _fill(b, b.k, b.v * 0.01)
    scale = 0.05
    clean, clean_lse = b.run(scale, window)
    place = n - 1 - window if T == 1 else n - T // 2 - 1   # just left of the window; seen by the later tokens
    k, v = b.k.copy(), b.v.copy()
    v[place] = np.resize([4e5, -3e5, 2.0], d)
    k[place] *= 1e4
    _fill(b, k, v)
    out, lse = b.run(scale, window)
    pos = n - T + np.arange(T)
    seen = (pos >= place) & ((pos < place + window) | (window == 0))
    not_seen = torch.from_numpy(~seen).cuda()
    assert (~seen).any() and seen.any() == (T > 1)
    assert torch.equal(out[not_seen], clean[not_seen]) and torch.equal(lse[not_seen], clean_lse[not_seen])


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("lens,news", [([3, 1, 40], [8, 5, 2]), ([3, 300, 0], [200, 150, 100])])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30])
def test_a_window_as_wide_as_any(name, lens, news, window):
    """A window past every length, beside tokens before the first key, is no window (few tokens and many)."""
    import torch
    b = Batch(91, lens, news, 2, 1, 64, 16, name)
    want, wlse = b.run(0.125)
    out, lse = b.run(0.125, window)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    b.check(window=window)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5])
def test_the_longest_sequence(name, T):
    """2^31 - 16 keys of one sequence, all in one page but the last 16.  Scores are 0 and values eighths from -7 to 8, so that the sums are
    exact in f32 while a warp's keys, times eight, are fewer than 2^24; the warps' and blocks' sums are joined in f32, at most
    12 + 152 roundings of 2^-24.  Then the last page's keys are 30 nats above the others: they make up the output but for
    2^31 / (16 e^30) = 1.3e-5 of values of at most 1.  Then a window over the last 40 keys."""
    import torch
    page, d, n = 16, 64, 2 ** 31 - 16
    pool = torch.zeros((2, qb.kv4_block_bytes(page, d)), dtype=torch.uint8, device="cuda")
    cache = qb.Kv4(pool, page, 1, d)
    rng = np.random.default_rng(93)
    v = rng.integers(-7, 8, (32, 1, d)) / 8
    v[:, :, ::32] = 1.0      # a group's extreme: the step is -1/8
    vt = torch.from_numpy(v.astype(np.float32)).cuda()

    def fill(k):
        kt = torch.from_numpy(np.broadcast_to(k, (32, 1, d)).astype(np.float32)).cuda().contiguous()
        qb.kv4_append(cache, kt, vt, _i32(np.arange(32)))
        back = torch.empty_like(vt)
        qb.kv4_read(cache, _i32(np.arange(32)), torch.empty_like(kt), back)
        assert torch.equal(back, vt)

    tables = torch.zeros((1, n // page), dtype=torch.int32, device="cuda")
    tables[0, -1] = 1
    seqs = qb.KvSeqs(tables, _i32([n]), q_start=_i32([0, T]))
    q = torch.ones((T, 1, d), dtype={"f32": torch.float32, "bf16": torch.bfloat16}[name], device="cuda")
    out, lse = torch.empty_like(q), torch.empty((T, 1), device="cuda")
    rounding = 164 * 2.0 ** -24 + OUT[name]
    fill(0.0)
    qb.kv4_attn(cache, q, seqs, 1.0, out, lse=lse)
    got = out.double().cpu().numpy()[:, 0]
    for j in range(T):
        keys = n - T + 1 + j
        want = (v[:16, 0].sum(0) * (n // page - 1) + v[16:32 - T + 1 + j, 0].sum(0)) / keys
        assert np.all(np.abs(got[j] - want) <= rounding)
        assert abs(float(lse[j]) - np.log(keys)) <= SUM * (1 + np.log(keys))
    k = np.zeros((32, 1, d))
    k[16:] = 30.0 / d
    fill(k)
    if T == 1:
        kb = torch.empty_like(vt)
        qb.kv4_read(cache, _i32(np.arange(32)), kb, torch.empty_like(vt))
        gap = float(kb[16].double().sum())
        qb.kv4_attn(cache, q, seqs, 1.0, out, lse=lse)
        assert np.all(np.abs(out.double().cpu().numpy()[0, 0] - v[16:, 0].mean(0)) <= 2 * (n - 16) / (16 * np.exp(gap)) + rounding + 2 * gap * SUM)
        assert abs(float(lse[0]) - (gap + np.log(16))) <= (n - 16) / (16 * np.exp(gap)) + SUM * (2 + gap) * 2
    fill(0.0)
    qb.kv4_attn(cache, q, seqs, 1.0, out, lse=lse, window=40)
    got = out.double().cpu().numpy()[:, 0]
    for j in range(T):
        places = np.arange(n - T + j - 39, n - T + j + 1, dtype=np.int64)
        rows = np.where(places >= n - 16, 16 + places % 16, places % 16)
        assert np.all(np.abs(got[j] - v[rows, 0].mean(0)) <= rounding)
        assert abs(float(lse[j]) - np.log(40)) <= SUM * 5


def test_calls_without_rows():
    """Every call through the binding with empty tensors: nothing changes, nothing is refused."""
    import torch
    b = Batch(95, [20, 0], [0, 0], 4, 2, 64, 16, "f32")
    page, npages, nrows, maxp = 16, b.pool.shape[0], 3, 4
    state = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, npages, npages, nrows, (nrows, maxp))]
    pages = qb.KvPages(page, *state)
    qb.kv_pages_reset(pages)
    before = [x.clone() for x in (*state, b.pool)]
    no, rows, q = _i32([]), torch.empty((0, 2, 64), device="cuda"), torch.empty((0, 4, 64), device="cuda")
    qb.kv4_append(b.cache, rows, rows, no)
    qb.kv4_read(b.cache, no, rows, rows)
    tables, lens = _i32(b.tables), _i32(b.lens)
    for seqs in (qb.KvSeqs(tables, lens, q_start=_i32([0, 0, 0])), qb.KvSeqs(tables, lens, rows=no), qb.KvSeqs(tables, lens, rows=no, q_start=_i32([0]))):
        qb.kv4_attn(b.cache, q, seqs, 0.125, torch.empty_like(q), lse=torch.empty((0, 4), device="cuda"))
    qb.kv_pages_extend(pages, no, no, no, no)
    status = _i32([5, 5])
    qb.kv_pages_extend(pages, _i32([0, 2]), _i32([0, 0]), no, status)
    assert status.tolist() == [0, 0]
    qb.kv_pages_fork(pages, b.pool, no, no, no)
    qb.kv_pages_free(pages, no)
    qb.kv_pages_copy(b.pool, npages, no, no)
    assert all(torch.equal(x, y) for x, y in zip((*state, b.pool), before))
    assert qb.q_device_status() == qb.QB_OK


@pytest.mark.parametrize("what", ["attn", "fork", "compact"])
def test_a_workspace_for_another_stream_is_not_memory_still_in_use_here(what, monkeypatch):
    """A block given back on the current stream, whose queued work still writes it, is not the workspace of a call on another stream."""
    import torch
    from block_quantized_weight_quantize_gb300 import kv4
    b = Batch(97, [40, 0], [1, 0], 4, 2, 64, 16, "f32")
    npages = b.pool.shape[0]
    state = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (1, npages, npages, 2, (2, 4))]
    pages = qb.KvPages(16, *state)
    qb.kv_pages_reset(pages)
    seqs = qb.KvSeqs(_i32(b.tables), _i32(b.lens), q_start=_i32(b.q_start))
    out, status, zero, one = torch.empty_like(b.q), _i32([5]), _i32([0]), _i32([1])
    side = torch.cuda.Stream()
    size = qb.kv4_attn_workspace_bytes(b.cache, b.q) if what == "attn" else qb.kv_pages_workspace_bytes(pages)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty(size, dtype=torch.uint8, device="cuda")
    where = block.data_ptr()
    torch.cuda._sleep(50_000_000)
    block.fill_(1)
    del block
    made, empty = [], torch.empty

    def note(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    with monkeypatch.context() as mp:
        mp.setattr(kv4.torch, "empty", note)
        if what == "attn":
            kv4.kv4_attn(b.cache, b.q, seqs, 0.125, out, stream=side)
        elif what == "fork":
            kv4.kv_pages_fork(pages, b.pool, zero, one, status, stream=side)
        else:
            kv4.kv_pages_compact(pages, b.pool, stream=side)
    assert len(made) == 1 and made[0].numel() == size and made[0].data_ptr() != where
    # and it is that stream's: given back, it goes to the next call there and to none here
    mine = made.pop().data_ptr()
    assert torch.empty(size, dtype=torch.uint8, device="cuda").data_ptr() != mine
    with torch.cuda.stream(side):
        again = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert again.data_ptr() == mine
    torch.cuda.synchronize()
    if what == "attn":
        want, _ = b.run(0.125)
        assert torch.equal(out, want)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("nh,nkv,d,lens,news,rel", [
    (4, 2, 64, [100, 40, 300], [60, 40, 200], 2.0 ** -10), (4, 1, 128, [900, 33], [50, 33], 2.0 ** -10), (6, 2, 96, [1500], [130], 2.0 ** -10),
    (8, 1, 128, [300, 17, 1000], [4, 1, 3], 2.0 ** -11), (4, 2, 256, [500], [120], 2.0 ** -11), (3, 3, 64, [700, 20], [2, 5], 2.0 ** -11)])
@pytest.mark.parametrize("kmul,window", [(1.0, 0), (6.0, 0), (1.0, 37)])
def test_half_precision_holds_its_accuracy(name, nh, nkv, d, lens, news, rel, kmul, window):
    """Rows of fewer than 2048 keys: queries and keys enter the scores without a rounding, so that a score is off by at most its
    magnitudes' sum times 2^-19 (f32 sums), lse by that and 2^-19 of its own parts, and an output by twice that relatively and `rel`:
    2^-11 for the probability times the step (few tokens), 2^-11 each for probability and value (many)."""
    b = Batch(d + nh, lens, news, nh, nkv, d, 16, name, kmul=kmul)
    scale = d ** -0.5
    out, lse = b.run(scale, window)
    want, wlse, zabs, mag = b.want(scale, window)
    off = zabs * SUM
    tol = (2 * off + rel + SUM)[..., None] * mag + OUT[name] * np.abs(want) + 2.0 ** -25 * (name == "f16")
    tol += len(b.v) * np.abs(b.v).max() * 2.0 ** -36
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= tol), np.max(err / tol)
    lerr, ltol = np.abs(lse.double().cpu().numpy() - wlse), off + SUM * (1 + np.abs(wlse))
    assert np.all(lerr <= ltol), np.max(lerr / ltol)
