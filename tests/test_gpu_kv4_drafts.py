"""Drafted trees as a server calls them: examples/kv4_decode.py checks a tree in one pass, and goes on from what stays."""
import pytest

import block_quantized_weight_quantize_gb300 as qb
from test_gpu_kv4_server import _example

pytestmark = pytest.mark.gpu


def test_the_example_checks_a_tree():
    """The accepted drafts are the tokens that the steps chose, and what follows them too.  33 tokens stay, as in the stepped
    sequence, on pages of 16: the first is shared, each sequence has two of its own.  The next token's outputs differ as a
    prompt's from its steps' (test_gpu_kv4_server.py): by 4-bit codes that move by one."""
    r = _example().drafts()
    assert r["kept"] == [0, 2, 4] and r["following"] == r["chosen"][3]
    assert r["lens"][:2] == [33, 33]
    assert r["pages held"] == 5
    assert r["tree against steps"] < 5e-3
    assert r["status"] == qb.QB_OK

