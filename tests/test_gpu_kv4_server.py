"""The products, the paged 4-bit cache and its pages together (examples/kv4_decode.py), and calls on a stream of their own."""
import importlib.util
import pathlib

import pytest

import block_quantized_weight_quantize_gb300 as qb

pytestmark = pytest.mark.gpu


def _example():
    path = pathlib.Path(__file__).resolve().parent.parent / "examples" / "kv4_decode.py"
    spec = importlib.util.spec_from_file_location("kv4_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example():
    """The prompt and the steps see the same keys through different orders of the sums; a difference in a key's last bits
    may move one of its 4-bit codes by one in the second layer, a 14th of its group's largest value: a few of 40 tokens'
    outputs by some 1e-3 at most.  Pages: 40 tokens are two full pages, shared, and one partly filled, copied.  In the
    end sequences of 50 and 50 tokens hold 2 + 2 + 2 pages; compacted, these are the first ones."""
    r = _example().run()
    assert r["prompt against steps"] < 5e-3
    assert r["pages a fork takes"] == 1
    assert r["fork differs"] == 0 and r["compacting changes"] == 0
    assert r["pages held"] == 6 and r["highest page held"] == 5
    assert r["pages free at the end"] == 64
    assert r["status"] == qb.QB_OK


@pytest.mark.parametrize("what", ["attn", "compact"])
def test_a_workspace_of_its_own_lives_as_long_as_its_stream_needs_it(what, monkeypatch):
    """A workspace that the binding makes for a call on another stream is not given out again while that stream runs."""
    import torch
    from block_quantized_weight_quantize_gb300 import kv4
    m = _example().Decoder()
    m.forward(torch.randn((20, 512), device="cuda"), [0], [20])
    q = torch.randn((1, 8, 64), device="cuda")
    out = torch.empty_like(q)
    seqs = qb.KvSeqs(m.pages.tables, m.pages.lens, torch.zeros(1, dtype=torch.int32, device="cuda"))
    made = []
    empty = torch.empty

    def note(*a, **kw):
        made.append(empty(*a, **kw))
        return made[-1]

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with monkeypatch.context() as mp:
        mp.setattr(kv4.torch, "empty", note)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # some 0.1 s
        if what == "attn":
            kv4.kv4_attn(m.caches[0], q, seqs, 0.125, out, stream=side)
        else:
            kv4.kv_pages_compact(m.pages, m.data, stream=side)
    assert len(made) == 1
    where, size = made[0].data_ptr(), made[0].numel()
    made.clear()
    later = torch.empty(size, dtype=torch.uint8, device="cuda")
    busy = not side.query()
    assert not busy or later.data_ptr() != where
    torch.cuda.synchronize()
    assert busy, "the stream was done before the check"
    assert qb.q_device_status() == qb.QB_OK
