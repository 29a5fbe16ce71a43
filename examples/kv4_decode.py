"""Two attention layers of a decoder on the paged 4-bit cache, as a server runs them: prompts, a fork, steps, a sequence
freed, the pool compacted.

    python examples/kv4_decode.py

Each layer's query, key and value products are one `q_matvec_many` per 16 tokens (Q8_0 weights), the new keys and values
go into the cache with `kv4_append`, `kv4_attn` reads it, and the output product closes the layer.  The pages are shared by
all layers: one `kv_pages_extend` a pass makes the room and gives the slots.  Weights and tokens are seeded random numbers.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import block_quantized_weight_quantize_gb300 as qb
from block_quantized_weight_quantize_gb300 import synth

HIDDEN, NH, NKV, D, LAYERS = 512, 8, 2, 64, 2
PAGE, NPAGES, NROWS, MAXP = 16, 64, 4, 16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Decoder:
    def __init__(self, seed: int = 0):
        rng = np.random.default_rng(seed)

        def weight(rows, K):
            return torch.from_numpy(synth.pack(synth.FMT_Q8_0, synth.draw(synth.FMT_Q8_0, rng, rows, K,
                                                                          d_range=(2e-4, 1e-3)))).cuda()

        self.rows = [NH * D, NKV * D, NKV * D]
        self.qkv = [[weight(r, HIDDEN) for r in self.rows] for _ in range(LAYERS)]
        self.o = [weight(HIDDEN, NH * D) for _ in range(LAYERS)]
        # the cache: every layer's pages in one allocation, one page table for all layers
        self.data = torch.empty((LAYERS, NPAGES, NKV * qb.kv4_block_bytes(PAGE, D)), dtype=torch.uint8, device="cuda")
        self.caches = [qb.Kv4(self.data[layer], PAGE, NKV, D) for layer in range(LAYERS)]
        self.pages = qb.KvPages(PAGE, i32([0]), *(torch.zeros(n, dtype=torch.int32, device="cuda")
                                                  for n in (NPAGES, NPAGES, NROWS, (NROWS, MAXP))))
        qb.kv_pages_reset(self.pages)
        self.work = torch.empty(qb.kv4_attn_workspace_bytes(self.caches[0], torch.empty(1, NH, D)), dtype=torch.uint8,
                                device="cuda")
        self.page_work = torch.empty(qb.kv_pages_workspace_bytes(self.pages), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(NROWS, dtype=torch.int32, device="cuda")

    def product(self, Ws, rows, x):
        outs = [torch.empty((x.shape[0], r), device="cuda") for r in rows]
        for c in range(0, x.shape[0], 16):
            xs = x[c:c + 16]
            work = torch.empty(qb.q_matvec_workspace_bytes(qb.Q8_0, x.shape[1], xs.shape[0]), dtype=torch.uint8, device="cuda")
            qb.q_matvec_many(qb.Q8_0, Ws, rows, x.shape[1], xs, [o[c:c + 16] for o in outs], work)
        return outs

    def attend(self, layer, q, seqs):
        out = torch.empty_like(q)
        qb.kv4_attn(self.caches[layer], q, seqs, D ** -0.5, out, workspace=self.work)
        return out

    def forward(self, x, rows, counts):
        """The new tokens x [sum(counts), HIDDEN] of the sequences `rows`, counts[i] each, through both layers."""
        slots = torch.empty(x.shape[0], dtype=torch.int32, device="cuda")
        qb.kv_pages_extend(self.pages, i32(rows), i32(counts), slots, self.status)
        if int(self.status[:len(rows)].min()) < 0:
            raise RuntimeError(qb.strerror(int(self.status[:len(rows)].min())))
        seqs = qb.KvSeqs(self.pages.tables, self.pages.lens, i32(rows), i32([0, *np.cumsum(counts)]))
        for layer in range(LAYERS):
            xn = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
            q, k, v = (y.view(x.shape[0], -1, D) for y in self.product(self.qkv[layer], self.rows, xn))
            qb.kv4_append(self.caches[layer], k, v, slots)
            x = x + self.product([self.o[layer]], [HIDDEN], self.attend(layer, q, seqs).view(x.shape[0], -1))[0]
        return x

    def fork(self, parents, children):
        qb.kv_pages_fork(self.pages, self.data, i32(parents), i32(children), self.status, self.page_work)

    def free(self, rows):
        qb.kv_pages_free(self.pages, i32(rows))

    def compact(self):
        qb.kv_pages_compact(self.pages, self.data, self.page_work)


def run():
    """What the walk through a server's calls shows, as numbers."""
    m = Decoder()
    tokens = torch.randn((96, HIDDEN), generator=torch.Generator().manual_seed(1)).cuda()
    first, second = tokens[:40], tokens[40:65]
    result = {}
    # two prompts in one pass, then the first one again token by token
    prompts = m.forward(torch.cat([first, second]), [0, 1], [40, 25])
    steps = torch.cat([m.forward(t[None], [2], [1]) for t in first])
    result["prompt against steps"] = float((prompts[:40] - steps).norm() / steps.norm())
    m.free([2])
    # a fork shares the full pages; given the same tokens it gives the same bits
    before = int(m.pages.nfree)
    m.fork([0], [2])
    result["pages a fork takes"] = before - int(m.pages.nfree)
    for t in tokens[65:75]:
        y = m.forward(t.expand(3, -1).contiguous(), [0, 1, 2], [1, 1, 1])
    result["fork differs"] = int((y[0] != y[2]).sum())
    # the second sequence ends, the pool is compacted, the others go on unmoved
    q = torch.randn((2, NH, D), generator=torch.Generator().manual_seed(2)).cuda()
    seqs = qb.KvSeqs(m.pages.tables, m.pages.lens, i32([0, 2]))
    m.free([1])
    old = [m.attend(layer, q, seqs) for layer in range(LAYERS)]
    m.compact()
    result["compacting changes"] = sum(int((m.attend(layer, q, seqs) != old[layer]).sum()) for layer in range(LAYERS))
    result["pages held"] = NPAGES - int(m.pages.nfree)
    result["highest page held"] = int(m.pages.tables.max())
    m.free([0, 2])
    result["pages free at the end"] = int(m.pages.nfree)
    result["status"] = qb.q_device_status()
    return result


if __name__ == "__main__":
    for name, value in run().items():
        print(f"{name}: {value}")
