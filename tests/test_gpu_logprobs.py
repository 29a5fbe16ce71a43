"""q_logprobs on the GPU against 64 bits.

Tolerances.  A term 2^d is off by the rounding of its difference and product (2^-23 of |d|, and |d| weighed by the
probabilities is E|d|, computed here) and by the exponential's 2^-22; a thread adds up to vocab / 256 + 16 of them one after
the other and then joins 13 levels: S is off relatively by A = (vocab / 256 + 32) 2^-24 + 2^-21 + 2^-22 E|d|.  So ln S is off by
A, a log probability by A, the rounding of (x - X) * scale and of the result (2^-22 of the two), lse likewise; T / S, which the
entropy takes from ln S, by 2 A E|d| more.  Places are whole numbers and equal."""
import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb

pytestmark = pytest.mark.gpu

F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    qb.lib()
    yield
    torch.cuda.synchronize()
    assert qb.q_device_status() == qb.QB_OK


def call(x, tokens=None, k=0, scale=1.0, stream=None):
    import torch
    n = x.shape[0]
    o = {"entropy": torch.full((n,), 9.0, device="cuda"), "lse": torch.full((n,), 9.0, device="cuda")}
    if tokens is not None:
        o["logprobs"] = torch.full(tokens.shape, 9.0, device="cuda")
    if k:
        o["top_tokens"], o["top_logprobs"] = torch.full((n, k), 9, dtype=torch.int32, device="cuda"), torch.full((n, k), 9.0, device="cuda")
    qb.q_logprobs(x, tokens=tokens, scale=scale, stream=stream, **o)
    torch.cuda.synchronize()
    return {a: b.cpu().numpy() for a, b in o.items()}


def check(x, tokens=None, k=0, scale=1.0, **kw):
    got = call(x, tokens, k, scale, **kw)
    xs = x.double().cpu().numpy()
    n, vocab = xs.shape
    scale = float(F32(scale))
    for i in range(n):
        row = xs[i]
        if np.isnan(row).any() or np.isposinf(row).any():
            for name, v in got.items():
                assert np.all(v[i] == -1) if name == "top_tokens" else np.isnan(v[i]).all(), name
            continue
        order = np.lexsort((np.arange(vocab), -row))[:k]
        if k:
            assert np.array_equal(got["top_tokens"][i], order), (i, got["top_tokens"][i], order)
        top = row.max()
        if np.isneginf(top):
            assert np.isneginf(got["lse"][i]) and got["entropy"][i] == 0
            if tokens is not None:
                assert np.isneginf(got["logprobs"][i]).all()
            if k:
                assert np.isneginf(got["top_logprobs"][i]).all()
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            d = (row - top) * scale
        e = np.exp(d)
        S = e.sum()
        p = e / S
        ed = float((p * np.where(p > 0, np.abs(d), 0)).sum()) * 1.4427
        a = (vocab / 256 + 32) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * ed
        lse = top * scale + np.log(S)
        assert abs(got["lse"][i] - lse) <= a + 2.0 ** -22 * (abs(top * scale) + abs(lse))
        h = np.log(S) - float((p * np.where(p > 0, d, 0)).sum())
        assert abs(got["entropy"][i] - h) <= a * (1 + 2 * ed) + 2.0 ** -22 * (np.log(S) + abs(h)), (i, got["entropy"][i], h)

        def near(g, places):
            for v, t in zip(g, places):
                w = d[t] - np.log(S) if 0 <= t < vocab else -np.inf
                with np.errstate(over="ignore"):
                    over = np.isneginf(F32(w))  # past f32's least number
                if over:
                    assert np.isneginf(v)
                else:
                    assert abs(v - w) <= a + 2.0 ** -22 * (abs(d[t]) + abs(w)), (i, v, w)

        if tokens is not None:
            near(got["logprobs"][i], tokens[i].cpu().numpy())
        if k:
            near(got["top_logprobs"][i], order)
    return got


def _type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def logits(seed, n, vocab, name="f32", spread=3.0):
    import torch
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((n, vocab)) * spread).astype(F32)).cuda().to(_type(name))


def given(seed, n, m, vocab):
    import torch
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.integers(0, vocab, (n, m)).astype(np.int32)).cuda()


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("n,vocab,k,m", [(1, 1, 1, 1), (3, 2, 2, 3), (2, 31, 31, 1), (5, 257, 64, 2), (2, 1000, 20, 0), (1, 2047, 64, 1), (1, 2049, 5, 1), (2, 4099, 33, 7),
                                         (1, 49152, 5, 1), (3, 40001, 64, 2), (700, 1111, 3, 1), (310, 9001, 20, 1)])
def test_sizes(name, n, vocab, k, m):
    """One token to long rows; rows that begin at any place of 16 bytes; one block a row and clusters of up to 16."""
    check(logits(vocab + k, n, vocab, name), given(k, n, m, vocab) if m else None, k, scale=1.0 if n % 2 else 0.7)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab,k,m", [(1, 1, 1), (3, 2, 0), (63, 32, 1), (515, 20, 1), (1024, 5, 0), (2100, 32, 2), (8192, 3, 1)])
def test_many_short_rows(name, vocab, k, m):
    """More rows than blocks run at once; the last ones masked, equal, rising, without a distribution."""
    import torch
    n = 640
    x = logits(vocab, n, vocab, name)
    x[-1] = -float("inf")
    x[-2] = 0.5
    x[-3] = torch.arange(vocab, device="cuda") * 0.01
    x[-4, vocab // 2] = float("nan")
    x[-5, vocab // 3] = float("inf")
    x[-6] = torch.finfo(x.dtype).min
    x[-7, 1:] = -float("inf")
    check(x, given(k, n, m, vocab) if m else None, k, scale=0.9)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("lead", [0, 1, 3, 7])
def test_strides_and_alignments(name, lead):
    """Rows inside a wider buffer that begins anywhere: values around them are never taken for logits."""
    import torch
    wide = torch.full((6, 5013), 1e4, device="cuda").to(_type(name))
    x = wide.flatten()[lead:lead + 5 * 5013 + 3001].as_strided((6, 3001), (5013, 1))
    x.copy_(logits(3, 6, 3001, name))
    check(x, given(1, 6, 2, 3001), 9)


def test_rows_further_apart_than_32_bits_count():
    import torch
    n, vocab, stride = 3, 5003, 2 ** 31 + 3
    wide = torch.empty(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = wide.as_strided((n, vocab), (stride, 1))
    x.copy_(logits(12, n, vocab, "bf16"))
    check(x, given(1, n, 2, vocab), 9)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "masked", "few", "lowest", "halves", "saw"])
def test_orders(name, kind):
    """Ties, sorted rows, rows with fewer tokens than alternatives, the type's lowest value as the mask."""
    import torch
    n, vocab, k = 3, 20011, 20
    t = torch.arange(vocab, device="cuda").float()
    lowest = torch.finfo(_type(name)).min
    x = {"equal": torch.zeros(vocab, device="cuda"), "rising": t * 1e-3, "falling": -t * 1e-3, "masked": torch.full((vocab,), -float("inf"), device="cuda"),
         "few": torch.full((vocab,), -float("inf"), device="cuda"), "lowest": torch.full((vocab,), lowest, device="cuda"),
         "halves": (t % 2), "saw": (t % 257) * 0.01}[kind].expand(n, -1).clone().to(_type(name))
    if kind == "few":
        x[0, 7] = 1.0
        x[1, [3, 19999, 20010, 0]] = torch.tensor([0.5, 0.5, -2.0, -0.0], device="cuda").to(_type(name))
        x[2, ::1500] = 2.0
    if kind == "lowest":
        x[0, [5, 17]] = 1.0
    check(x, given(2, n, 3, vocab), k)
    check(x, None, 64)
    check(x.expand(3, -1).repeat(110, 1)[:, :3000].contiguous(), None, k)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(1, 200003), (700, 30000), (640, 8000)])
def test_the_largest_in_few_threads(name, n, vocab):
    """Large logits in runs of 16 bytes that recur with every 256th (64th) run: a few threads of each block have them all."""
    import torch
    x = logits(11, n, vocab, name, 0.1)
    per = 4 if name == "f32" else 8
    run = torch.arange(vocab, device="cuda") // per
    x += (5.0 * ((run % 256 < 70) | (run % 64 < 5))).to(x.dtype)
    rows = [0, n // 2, n - 1]
    got = {k: call(x, None, k) for k in (5, 32, 64)}
    for k, g in got.items():
        for i in rows:
            row = x[i].double().cpu().numpy()
            assert np.array_equal(g["top_tokens"][i], np.lexsort((np.arange(vocab), -row))[:k])


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(2, 41549), (50, 4289), (700, 4289), (3, 128256), (650, 70000)])
@pytest.mark.parametrize("kind", ["masked", "levels", "late"])
def test_many_equal_logits(name, n, vocab, kind):
    """Rows of which almost all is forbidden, rows of a few different values, and equal ones that come late or between larger ones:
    places by value, then in order, whichever block and pass they come from."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(vocab + n)
    x = logits(13, n, vocab, name)
    u = torch.rand((n, vocab), device="cuda", generator=g)
    if kind == "masked":
        x[u < 0.999] = -float("inf")
    elif kind == "levels":
        x = (u * 3).floor().to(_type(name))
    else:
        x = torch.where(u < 0.0003, 3.0, torch.where(torch.arange(vocab, device="cuda") > vocab * 0.7, 1.0, 0.0)).to(_type(name))
    rows = [0, n // 2, n - 1]
    for k in (1, 20, 32, 64):
        got = call(x, None, k)
        for i in rows:
            row = x[i].double().cpu().numpy()
            assert np.array_equal(got["top_tokens"][i], np.lexsort((np.arange(vocab), -row))[:k]), (k, i)


def test_signed_zeros_are_equal():
    import torch
    x = torch.full((1, 100), -1.0, device="cuda")
    x[0, 40], x[0, 60] = -0.0, 0.0
    assert call(x, None, 2)["top_tokens"].tolist() == [[40, 60]]


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_rows_without_a_distribution(name):
    """A NaN or +infinity spoils its own row only; tokens outside the vocabulary have no probability."""
    import torch
    for vocab in (300, 30000):
        x = logits(4, 6, vocab, name)
        x[1, 5] = float("nan")
        x[3, vocab - 1] = float("inf")
        x[4] = -float("inf")
        tokens = torch.tensor([[0, -1, vocab, 2 ** 31 - 1, -2 ** 31]] * 6, dtype=torch.int32, device="cuda")
        check(x, tokens, 7)


@pytest.mark.parametrize("spread", [1e-3, 40.0, 3000.0, 1e30])
def test_flat_and_sharp_rows(spread):
    """From the uniform distribution to one token with all of it; the entropy is never negative."""
    got = check(logits(5, 4, 30011, "f32", spread), given(5, 4, 3, 30011), 10)
    assert (got["entropy"] >= 0).all()


def test_a_rising_row_moves_the_reference():
    """Each element is far above the one before it: the reference moves at each of a thread's elements."""
    import torch
    x = (torch.arange(30000, device="cuda").float() * 0.05)[None].repeat(2, 1)
    check(x, given(1, 2, 4, 30000), 64)
    check(x.flip(1).contiguous(), given(1, 2, 4, 30000), 64)


@pytest.mark.parametrize("scale", [2.0 ** -20, 0.3, 2.0 ** 20])
def test_scales(scale):
    check(logits(6, 2, 5000), given(6, 2, 3, 5000), 5, scale=scale)


def test_single_outputs():
    """Each output by itself is what it is with the others."""
    import torch
    x, tokens = logits(7, 3, 20000), given(7, 3, 2, 20000)
    want = call(x, tokens, 6)
    for name, shape, typ in (("entropy", (3,), torch.float32), ("lse", (3,), torch.float32), ("top_tokens", (3, 6), torch.int32), ("top_logprobs", (3, 6), torch.float32)):
        o = torch.zeros(shape, dtype=typ, device="cuda")
        qb.q_logprobs(x, **{name: o})
        assert np.array_equal(o.cpu().numpy(), want[name])
    o = torch.zeros((3, 2), device="cuda")
    qb.q_logprobs(x, tokens=tokens, logprobs=o)
    assert np.array_equal(o.cpu().numpy(), want["logprobs"])


def test_the_same_bits_each_time_on_any_stream_and_from_a_graph():
    import torch
    for n, vocab in ((2, 49152), (400, 3001)):
        x, tokens = logits(8, n, vocab, "bf16"), given(8, n, 1, vocab)
        want = call(x, tokens, 12)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for stream in (None, side):
            got = call(x, tokens, 12, stream=stream)
            assert all(np.array_equal(got[a], want[a]) for a in want)
        y = torch.zeros_like(x)
        o = {a: torch.zeros(b.shape, dtype=torch.int32 if b.dtype == np.int32 else torch.float32, device="cuda") for a, b in want.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            qb.q_logprobs(y, tokens=tokens, **o)
        y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(o[a].cpu().numpy(), want[a]) for a in want)


def test_refusals():
    import torch
    x = logits(9, 2, 50)
    f = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for kw in (dict(tokens=i(2, 1)), dict(logprobs=f(2, 1)), dict(tokens=i(3, 1), logprobs=f(3, 1)), dict(tokens=i(2, 1), logprobs=f(2, 2)), dict(entropy=f(3)), dict(lse=f(2).cpu()),
               dict(entropy=f(2).double()), dict(top_tokens=i(2, 3), top_logprobs=f(2, 4)), dict(top_tokens=i(2)), dict(top_logprobs=f(1, 3)), dict(tokens=f(2, 1), logprobs=f(2, 1))):
        with pytest.raises(ValueError):
            qb.q_logprobs(x, **kw)
    for kw in (dict(top_tokens=i(2, 51)), dict(top_tokens=i(2, 65)), dict(scale=0.0, lse=f(2)), dict(scale=float("nan"), lse=f(2))):
        with pytest.raises(qb.QbError):
            qb.q_logprobs(x, **kw)
    for bad in (x.double(), x[0], x.t(), x.cpu(), x[:, ::2]):
        with pytest.raises(ValueError):
            qb.q_logprobs(bad, lse=f(2))
    qb.q_logprobs(x[:0], lse=f(0))
