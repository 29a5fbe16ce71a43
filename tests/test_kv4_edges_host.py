"""The paged 4-bit cache at its edges, on a host without a GPU: what calls without work, orders of kernels and index
arithmetic have to keep to."""
import ctypes
import pathlib
import re
import shutil
import subprocess

import pytest

import block_quantized_weight_quantize_gb300 as qb
from block_quantized_weight_quantize_gb300 import kv4
from test_kv4_host import A, _cache, _pages, _seqs

CSRC = pathlib.Path(__file__).resolve().parent.parent / "block_quantized_weight_quantize_gb300" / "csrc"
TOP = 2 ** 31


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    """The functions of qb_kv_index.h and qb_fault.h as a host library, every signed overflow an abort."""
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("index")
    (d / "i.cpp").write_text("""#include "qb_fault.h"
#include "qb_kv_index.h"
extern "C" int reported(int word) { return qb::fault_reported(word); }
extern "C" int status(int bit) { return qb::fault_status(bit); }
extern "C" long long room(long long c, long long first, long long n) { return qb::kv_slots_room(c, first, n); }
extern "C" int parts(int len, int size) { return qb::kv_parts(len, size); }
extern "C" int first_seen(int pos, int window) { return qb::kv_first_seen(pos, window); }
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", str(CSRC), "-I", str(CSRC.parent.parent / "include"), str(d / "i.cpp"),
                    "-o", str(d / "i.so")], check=True)
    lib = ctypes.CDLL(str(d / "i.so"))
    lib.room.argtypes, lib.room.restype = [ctypes.c_longlong] * 3, ctypes.c_longlong
    return lib


@pytest.mark.parametrize("count", [0, 1, 31, 32, 100, TOP - 33, TOP - 32, TOP - 31, TOP - 1])
@pytest.mark.parametrize("first", [0, 1, 49, 50, 51, TOP - 1, (TOP - 1) * (1 << 20)])
def test_slots_of_a_request_stay_in_their_array(index, count, first):
    """Whatever a request's count and place: the entries first .. first + room - 1 are in the array, and all of the request's that are."""
    for nslots in (0, 1, 50, TOP - 1, TOP * 8):
        room = index.room(count, first, nslots)
        assert room == len(range(first, min(first + count, nslots)))


@pytest.mark.parametrize("file,kernel", [("qb_kv.cu", "kv_cache_rows_kernel"), ("qb_kv_pages.cu", "kv_pages_copy_kernel")])
def test_writers_of_a_key_cache_let_no_kernel_start_early(file, kernel):
    """kv_scores reads its first key tiles before it waits for the kernel before it, so no kernel that may write a key cache
    starts its successor early."""
    text = (CSRC / file).read_text()
    body = re.search(r"__global__[^;{]*\b%s\(.*?\n}\n" % kernel, text, re.S).group(0)
    assert "pdl_wait();" in body and "pdl_launch_dependents();" not in body


@pytest.mark.parametrize("window", [0, 1, 2, 50, TOP - 18, TOP - 17, TOP - 1])
def test_first_key_seen(index, window):
    """Places from 2^24 tokens before the first key up to the last key of the longest table row."""
    for pos in (-(1 << 24), -5, -1, 0, 1, 48, 49, 50, 51, TOP - 19, TOP - 18, TOP - 17):
        assert index.first_seen(pos, window) == (max(0, pos - window + 1) if window else 0)


def test_parts_of_a_length(index):
    for n in (0, 1, 31, 32, 33, 64, TOP - 64, TOP - 33, TOP - 32, TOP - 31, TOP - 16, TOP - 1):
        assert index.parts(n, 32) == -(-n // 32)


def test_calls_without_rows_take_arrays_without_an_address():
    """An empty tensor's address is NULL.  Nothing else about the call may be wrong."""
    c, p, s, f = _cache(), _pages(), _seqs(q_start=A), kv4._c
    ca, pa, sa = (ctypes.addressof(x) for x in (c, p, s))
    assert f.kv4_append(ca, 0, None, 128, None, 128, None, 0, None) == qb.QB_OK
    assert f.kv4_read(ca, 0, None, 0, None, 128, None, 128, None) == qb.QB_OK
    assert f.kv4_attn(ca, sa, 0, None, 256, 0, 4, 1.0, 0, None, 256, None, None, 0, None) == qb.QB_OK
    none = _seqs(nseq=0)
    na = ctypes.addressof(none)
    assert f.kv4_attn(ca, na, 0, None, 256, 0, 4, 1.0, 0, None, 256, None, None, 0, None) == qb.QB_OK
    assert f.kv_pages_extend(pa, None, None, 0, None, 0, None, None) == qb.QB_OK
    assert f.kv_pages_fork(pa, A, 1, 64, None, None, 0, None, None, 0, None) == qb.QB_OK
    assert f.kv_pages_free(pa, None, 0, None) == qb.QB_OK
    assert f.kv_pages_copy(A, 1, 8, 64, None, None, 0, None) == qb.QB_OK
    # tokens without a sequence, and what is wrong without rows too
    none.q_start = A
    assert f.kv4_attn(ca, na, 0, A, 256, 3, 4, 1.0, 0, A, 256, None, A, 1 << 30, None) == qb.QB_E_ARG
    assert f.kv4_append(ca, 7, None, 128, None, 128, None, 0, None) == qb.QB_E_ARG
    assert f.kv4_attn(ca, sa, 0, None, 256, 0, 3, 1.0, 0, None, 256, None, None, 0, None) == qb.QB_E_ARG
    assert f.kv_pages_fork(pa, None, 1, 64, None, None, 0, None, None, 0, None) == qb.QB_E_ARG
    # slots without an address only where there are none
    assert f.kv_pages_extend(pa, A, A, 1, None, 5, A, None) == qb.QB_E_ARG
    bad = _cache(page=24)
    assert f.kv4_append(ctypes.addressof(bad), 0, None, 128, None, 128, None, 0, None) == qb.QB_E_ARG


class _On:
    """A tensor's outside: on device `at`, at an address that nothing reads."""

    def __init__(self, at, shape, dtype):
        import torch
        self.like, self.at, self.dtype, self.shape = torch.empty(shape, dtype=dtype, device="meta"), at, dtype, torch.Size(shape)

    def __getattr__(self, name):
        return getattr(self.like, name)

    def get_device(self):
        return self.at

    def data_ptr(self):
        return A


@pytest.fixture
def calls(monkeypatch):
    """The entry points that a call reaches, none of them made; device 0 is the current one."""
    made = []

    class Entries:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or qb.QB_OK

    monkeypatch.setattr(kv4, "_c", Entries())
    monkeypatch.setattr(kv4, "_current_device", lambda: 0)
    monkeypatch.setattr(kv4, "_raw_stream", lambda dev: 0)
    return made


def _everything(at):
    """Every call of the binding with tensors where `at(name)` says."""
    import torch
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32

    def t(name, shape, dtype=i32):
        return _On(at(name), shape, dtype)

    bb = 64 * 16 // 2 * 2 + 64 * 16 // 16 * 2
    c = kv4._CKv4(A, 8, 16, 2, 64)
    cache = object.__new__(kv4.Kv4)
    cache.data, cache.page, cache.nkv, cache.d, cache.dev, cache.c, cache.ref = t("data", (8, 2 * bb), u8), 16, 2, 64, at("data"), c, ctypes.addressof(c)
    rows, q, lse, ws = ((3, 2, 64), (3, 4, 64), (3, 4), (1 << 20,))

    def seqs():
        return kv4.KvSeqs(t("tables", (3, 4)), t("lens", (3,)), t("rows", (3,)), t("q_start", (4,)))

    def pages():
        return kv4.KvPages(16, t("nfree", (1,)), t("free", (8,)), t("refs", (8,)), t("lens", (3,)), t("tables", (3, 4)))

    def pool():
        return t("pool", (2, 8, 64), u8)

    return {
        "kv4_append": lambda: kv4.kv4_append(cache, t("k", rows, f32), t("v", rows, f32), t("slots", (3,))),
        "kv4_read": lambda: kv4.kv4_read(cache, t("slots", (3,)), t("k", rows, f32), t("v", rows, f32)),
        "kv4_attn": lambda: kv4.kv4_attn(cache, t("q", q, f32), seqs(), 1.0, t("out", q, f32), t("lse", lse, f32), workspace=t("ws", ws, u8)),
        "kv_pages_reset": lambda: kv4.kv_pages_reset(pages()),
        "kv_pages_extend": lambda: kv4.kv_pages_extend(pages(), t("rows", (3,)), t("counts", (3,)), t("slots", (9,)), t("status", (3,))),
        "kv_pages_fork": lambda: kv4.kv_pages_fork(pages(), pool(), t("parents", (1,)), t("children", (1,)), t("status", (1,)), t("ws", ws, u8)),
        "kv_pages_free": lambda: kv4.kv_pages_free(pages(), t("rows", (3,))),
        "kv_pages_compact": lambda: kv4.kv_pages_compact(pages(), pool(), t("ws", ws, u8)),
        "kv_pages_copy": lambda: kv4.kv_pages_copy(pool(), 8, t("src", (2,)), t("dst", (2,))),
    }


USES = {"kv4_append": "data k v slots", "kv4_read": "data slots k v", "kv4_attn": "data q tables lens rows q_start out lse ws",
        "kv_pages_reset": "nfree free refs lens tables", "kv_pages_extend": "refs rows counts slots status", "kv_pages_fork": "refs pool parents children status ws",
        "kv_pages_free": "refs rows", "kv_pages_compact": "refs pool ws", "kv_pages_copy": "pool src dst"}


@pytest.mark.parametrize("call", sorted(USES))
def test_tensors_lie_on_the_current_device(calls, call):
    """On device 0, the current one, the call is made; all on device 1, or any one tensor there or in host memory, and nothing is."""
    _everything(lambda name: 0)[call]()
    assert calls == [call]
    calls.clear()
    with pytest.raises(ValueError, match="current device"):
        _everything(lambda name: 1)[call]()
    for one in USES[call].split():
        with pytest.raises(ValueError, match="cuda:"):
            _everything(lambda name: int(name == one))[call]()
        if one != "data":  # a cache refuses host memory itself
            with pytest.raises(ValueError, match="device memory"):
                _everything(lambda name: -int(name == one))[call]()
    assert calls == []


def test_every_kind_of_fault_is_reported(index):
    """A word with both kinds gives two reports, the given-up wait first; what one call reports is all that it clears."""
    reports = []
    word = 3
    for _ in range(3):
        bit = index.reported(word)
        reports.append(index.status(bit))
        word &= ~bit
    assert reports == [qb.QB_E_DEVICE, qb.QB_E_INDEX, qb.QB_OK] and word == 0
    assert index.status(index.reported(2)) == qb.QB_E_INDEX and index.status(index.reported(1)) == qb.QB_E_DEVICE
    text = (CSRC / "qb_api.cu").read_text()
    body = text[text.index("int q_device_status("):]
    body = body[:body.index("\n}\n")]
    assert "fault_clear_kernel" in body and "cudaMemcpyToSymbol" not in body    # no bit is overwritten
