"""Drafted trees, sinks and log probabilities on a host without a GPU: which keys a token sees (the index arithmetic of the
kernels, as a host library), and argument checks that answer before any CUDA call."""
import ctypes
import pathlib
import random
import shutil
import subprocess

import numpy as np
import pytest

import block_quantized_weight_quantize_gb300 as qb
from block_quantized_weight_quantize_gb300 import kv4
from test_kv4_host import A, ODD, _cache, _pages, _seqs

CSRC = pathlib.Path(__file__).resolve().parent.parent / "block_quantized_weight_quantize_gb300" / "csrc"
TOP = 2 ** 31


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    """The functions of qb_kv_index.h as a host library, every signed overflow an abort."""
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("index")
    (d / "i.cpp").write_text("""#include "qb_kv_index.h"
using namespace qb;
extern "C" unsigned range_word(int lo, int hi, int k0) { return kv_range_word(lo, hi, k0); }
extern "C" unsigned bits_at(const unsigned *m, int words, int at) { return kv_bits_at(m, words, at); }
// 0: tree, 1: causal
extern "C" void seen(const unsigned *mask, int words, int T, int j, int len, int window, int sinks, int k0, int n, unsigned *out, int *sight) {
    const int base = len - T;
    KvSight s = mask ? kv_tree_sight(mask, words, T, base, window) : KvSight{kv_first_seen(base + j, window), base + j, kKvNoKey};
    sight[0] = s.lo; sight[1] = s.hi; sight[2] = s.dlo;
    for (int i = 0; i < n; ++i) out[i] = kv_seen_word(s, window ? sinks : 0, mask, words, base, len, k0 + 32 * i);
}
extern "C" void parts(int first, int sinks, int size, int *out) { const KvParts p = kv_sink_parts(first, sinks, size); out[0] = p.hole; out[1] = p.jump; }
extern "C" int part(int u, int hole, int jump) { return kv_part(u, hole, jump); }
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", str(CSRC), str(d / "i.cpp"), "-o", str(d / "i.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "i.so"))
    lib.range_word.restype = lib.bits_at.restype = ctypes.c_uint
    return lib


def _seen(index, marks, words, T, j, len_, window, sinks, k0, n):
    out, sight = (ctypes.c_uint * n)(), (ctypes.c_int * 3)()
    mask = None if marks is None else (ctypes.c_uint * words)(*[marks >> 32 * w & 0xFFFFFFFF for w in range(words)])
    index.seen(mask, words, T, j, len_, window, sinks, k0, n, out, sight)
    return {k0 + 32 * i + b for i in range(n) for b in range(32) if out[i] >> b & 1}


def _want(marks, words, T, j, len_, window, sinks):
    base = len_ - T
    if marks is None:
        keys = list(range(max(0, base + j + 1)))
    else:
        keys = list(range(max(0, base))) + [base + i for i in range(min(T, 32 * words)) if marks >> i & 1 and base + i >= 0]
    if window:
        keys = sorted(set(keys[-window:]) | {k for k in keys if k < sinks})
    return set(keys)


def test_words_of_a_range(index):
    for lo, hi, k0 in [(0, -1, 0), (0, 0, 0), (0, 31, 0), (5, 40, 32), (33, 33, 32), (64, 70, 32), (0, 10, 32), (TOP - 1, TOP - 2, 0), (0, TOP - 1, TOP - 32), (3, 2, 0)]:
        assert index.range_word(lo, hi, k0) == sum(1 << i for i in range(32) if lo <= k0 + i <= hi)


def test_bits_at_any_place(index):
    m = (ctypes.c_uint * 2)(0x80000001, 0xDEADBEEF)
    v = 0x80000001 | 0xDEADBEEF << 32
    for at in range(-70, 140):
        assert index.bits_at(m, 2, at) == ((v << 200) >> (at + 200)) & 0xFFFFFFFF


def test_what_a_token_sees(index):
    r = random.Random(5)
    for _ in range(4000):
        words = r.choice((1, 1, 2, 3))
        T, len_ = r.randint(1, 40 * words), r.randint(0, 150)
        window, sinks = r.choice((0, 0, 1, 2, 5, 40, 200, TOP - 1)), r.choice((0, 1, 4, 33, 90, 500, TOP - 1))
        marks = r.choice((None, 0, r.getrandbits(32 * words), r.getrandbits(32 * words), r.getrandbits(32 * words) & r.getrandbits(32 * words)))
        j = r.randrange(T)
        got = _seen(index, marks, words, T, j, len_, window, sinks, 0, 6)
        assert got == _want(marks, words, T, j, len_, window, sinks), (marks, words, T, j, len_, window, sinks)


def test_what_a_token_sees_at_the_end_of_the_range(index):
    """The longest sequences: no arithmetic past 2^31, the last keys right."""
    len_ = TOP - 16
    k0 = (len_ - 64) // 32 * 32
    for window in (0, 1, 20, TOP - 1):
        for marks in (None, 0b1011, 0):
            got = _seen(index, marks, 1, 4, 3, len_, window, TOP - 1 if window == TOP - 1 else 3, k0, 3)
            base = len_ - 4
            keys = [k for k in range(k0, k0 + 96) if k < base] + [base + i for i in range(4) if (marks is None or marks >> i & 1)]
            if window and window < 1000:
                keys = keys[-window:]
            assert got == set(keys)


def test_parts_of_an_item_cover_the_sinks_and_the_window(index):
    r = random.Random(6)
    for _ in range(2000):
        size = r.choice((32, 128))
        first, sinks, more = r.randint(0, 3000), r.choice((0, 1, 31, 32, 33, 500, 5000, TOP - 1)), r.randint(1, 500)
        out = (ctypes.c_int * 2)()
        index.parts(first, sinks, size, out)
        end = -(-(first + more) // size)
        parts = [index.part(u, out[0], out[1]) for u in range(out[0], end)]
        assert parts == sorted(set(parts))
        assert set(parts) == {k // size for k in range(first + more) if k >= first or k < sinks} | set(range(first // size, end))


def test_attention_arguments():
    c = ctypes.addressof(k := _cache())
    s = ctypes.addressof(t := _seqs())
    need = kv4._c.kv4_attn_workspace_bytes(c, 4)

    def sinks(window=4, sinks=2, scale=1.0, q=A, wb=need):
        return kv4._c.kv4_attn_sinks(c, s, 0, q, 256, 3, 4, scale, window, sinks, A, 256, None, A, wb, None)

    def tree(window=0, sinks=0, masks=A, words=1, q=A, ntok=3):
        return kv4._c.kv4_attn_tree(c, s, 0, q, 256, ntok, 4, 1.0, window, sinks, masks, words, A, 256, None, A, need, None)

    for bad in (dict(window=-1), dict(sinks=-1), dict(scale=float("nan")), dict(q=ODD), dict(wb=need - 1)):
        assert sinks(**bad) == qb.QB_E_ARG, bad
    for bad in (dict(window=-1), dict(sinks=-1), dict(masks=None), dict(masks=4097), dict(words=0), dict(words=33), dict(q=None), dict(ntok=4)):
        assert tree(**bad) == qb.QB_E_ARG, bad
    assert k is not None and t is not None


def test_tree_arguments():
    f = kv4._c

    def masks(parents=A, ntok=3, q_start=A, nseq=2, m=A, words=1, depth=None):
        return f.kv_tree_masks(parents, ntok, q_start, nseq, m, words, depth, None)

    def accept(parents=A, tokens=A, targets=A, ntok=3, q_start=A, nseq=2, keep=A, nkeep=A, next_=A):
        return f.kv_tree_accept(parents, tokens, targets, ntok, q_start, nseq, keep, nkeep, next_, None)

    for bad in (dict(parents=None), dict(parents=4097), dict(ntok=-1), dict(ntok=(1 << 20) + 1), dict(nseq=0), dict(nseq=-1), dict(q_start=None), dict(q_start=4098),
                dict(m=None), dict(m=4098), dict(words=0), dict(words=33), dict(depth=4097)):
        assert masks(**bad) == qb.QB_E_ARG, bad
    assert masks(ntok=0, parents=None, m=None) == qb.QB_OK and masks(ntok=0, nseq=0, parents=None, m=None) == qb.QB_OK
    for bad in (dict(parents=None), dict(tokens=None), dict(targets=4097), dict(ntok=-1), dict(nseq=0), dict(q_start=None), dict(keep=None), dict(nkeep=None),
                dict(next_=None), dict(nkeep=4097)):
        assert accept(**bad) == qb.QB_E_ARG, bad
    assert accept(ntok=0, nseq=0, parents=None, tokens=None, targets=None, keep=None, nkeep=None, next_=None) == qb.QB_OK


def test_keep_arguments():
    p = ctypes.addressof(good := _pages())

    def keep(pages=p, data=A, layers=1, nkv=2, d=64, rows=A, q_start=A, keep=A, nkeep=A, ntok=5, n=2, status=A):
        return kv4._c.kv4_keep(pages, data, layers, nkv, d, rows, q_start, keep, nkeep, ntok, n, status, None)

    for bad in (dict(data=None), dict(data=ODD), dict(layers=0), dict(layers=65536), dict(nkv=0), dict(nkv=1025), dict(d=60), dict(d=264), dict(rows=4097), dict(q_start=None),
                dict(keep=None), dict(keep=4097), dict(nkeep=None), dict(ntok=-1), dict(ntok=TOP), dict(n=-1), dict(n=5), dict(status=None),
                dict(pages=ctypes.addressof(b := _pages(page=20)))):
        assert keep(**bad) == qb.QB_E_ARG, bad
    assert keep(n=0, rows=None, q_start=None, keep=None, nkeep=None, ntok=0, status=None) == qb.QB_OK
    assert good is not None and b is not None


def test_logprobs_arguments():
    def call(type_=0, x=A, stride=100, n=3, vocab=100, scale=1.0, tokens=A, m=1, logp=A, ent=A, lse=A, k=5, tt=A, tl=A):
        return kv4._c.q_logprobs(type_, x, stride, n, vocab, scale, tokens, m, logp, ent, lse, k, tt, tl, None)

    for bad in (dict(type_=3), dict(x=None), dict(x=4097), dict(x=4098), dict(type_=1, x=4097), dict(stride=99), dict(stride=(1 << 40) + 1), dict(n=-1), dict(n=(1 << 26) + 1),
                dict(vocab=0), dict(vocab=(1 << 24) + 1, stride=1 << 25), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(tokens=None), dict(logp=None), dict(tokens=4097), dict(m=-1), dict(m=1025), dict(ent=4097), dict(lse=4098), dict(k=-1), dict(k=65),
                dict(k=8, vocab=7, stride=7), dict(tt=4097), dict(tl=4099)):
        assert call(**bad) == qb.QB_E_ARG, bad
    assert call(n=0, x=None, tokens=None, logp=None) == qb.QB_OK


def test_binding_refuses_what_does_not_fit():
    import torch
    i, f = torch.zeros(4, dtype=torch.int32), torch.zeros((4, 9))
    for call in (lambda: qb.kv_tree_masks(i, torch.zeros((4, 1), dtype=torch.int32)), lambda: qb.kv_tree_accept(i, i, i, i, i, i), lambda: qb.q_logprobs(f),
                 lambda: qb.q_logprobs(f[0])):
        with pytest.raises(ValueError):
            call()
    assert np.iinfo(np.int32).max == TOP - 1
