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
    """The functions of qb_kv_index.h as a host library, every signed overflow an abort."""
    if not shutil.which("g++"):
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("index")
    (d / "i.cpp").write_text("""#include "qb_kv_index.h"
extern "C" long long room(long long c, long long first, long long n) { return qb::kv_slots_room(c, first, n); }
extern "C" int parts(int len, int size) { return qb::kv_parts(len, size); }
extern "C" int first_seen(int pos, int window) { return qb::kv_first_seen(pos, window); }
""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-ftrapv", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", str(CSRC), str(d / "i.cpp"),
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
