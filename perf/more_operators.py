"""Serving with drafted tokens on the paged 4-bit key/value cache: what the operators compute, in plain torch, and the cases they are timed on.

`kv4_attn_tree`: attention of drafted trees (a token sees what the cache held before the drafts, and the drafts that its mask marks), `kv4_attn_sinks`: causal
attention of the last `window` keys and a sequence's first few; `q_logprobs`: log probabilities of given tokens, entropy and the top alternatives from a row of
logits; `kv_tree_masks`, `kv_tree_accept` and `kv4_keep`: a tree's masks and depths, the path that the target's tokens take through it, and that path's rows moved
together in the cache, the other drafts' places and pages given back.

The cache holds, per page and key head, one block of bytes: the keys' codes, the keys' steps, the values' codes, the values' steps.  A row (one token, one head) of
d elements is stored as dp (d rounded up to 64, 128 or 256, the rest zeros) 4-bit codes with one f16 step per 32 of them; an element is (code - 8) * step.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a chat's first drafts on a small model with 9 query and 3 key heads: latency
        {"name": "tree, one short sequence", "op": "attn", "tree": True, "nseq": 1, "lo": 61, "hi": 61, "t": 8, "nh": 9, "nkv": 3, "d": 64,
         "page": 16, "type": "f32", "window": 0, "sinks": 0, "mix": 1},
        # the ordinary step of a server that drafts: a batch of unequal lengths, trees of up to 16 tokens
        {"name": "tree, a batch", "op": "attn", "tree": True, "nseq": 32, "lo": 1, "hi": 4096, "t": 16, "nh": 32, "nkv": 8, "d": 128,
         "page": 16, "type": "bf16", "window": 0, "sinks": 0, "mix": 2},
        # few sequences, for which wide trees are worth their products
        {"name": "tree, wide trees", "op": "attn", "tree": True, "nseq": 12, "lo": 500, "hi": 6000, "t": 64, "nh": 32, "nkv": 8, "d": 128,
         "page": 64, "type": "f16", "window": 0, "sinks": 0, "mix": 3},
        # wide heads shared eight ways, in f32, a sliding window and sinks under the trees
        {"name": "tree, wide heads, window", "op": "attn", "tree": True, "nseq": 9, "lo": 2000, "hi": 12000, "t": 21, "nh": 16, "nkv": 2, "d": 256,
         "page": 32, "type": "f32", "window": 4096, "sinks": 4, "mix": 4},
        # the step of a batch that streams on: 64 sequences, most of them longer than the window, one still empty
        {"name": "sinks, a batch's step", "op": "attn", "tree": False, "nseq": 64, "lo": 0, "hi": 8192, "t": 1, "nh": 32, "nkv": 8, "d": 128,
         "page": 16, "type": "f32", "window": 2048, "sinks": 4, "mix": 5},
        # one long stream with a wide window: the key axis has to be split
        {"name": "sinks, one long sequence", "op": "attn", "tree": False, "nseq": 1, "lo": 131071, "hi": 131071, "t": 1, "nh": 32, "nkv": 8, "d": 128,
         "page": 64, "type": "bf16", "window": 16384, "sinks": 100, "mix": 6},
        # a prompt's chunk over what is cached already
        {"name": "sinks, a prompt's chunk", "op": "attn", "tree": False, "nseq": 1, "lo": 8192, "hi": 8192, "t": 2048, "nh": 32, "nkv": 8, "d": 128,
         "page": 64, "type": "bf16", "window": 1024, "sinks": 4, "mix": 7},
        # one step of one sequence on the small model's vocabulary: latency
        {"name": "logprobs, one token", "op": "logprobs", "n": 1, "vocab": 49152, "type": "f32", "k": 5, "m": 1, "scale": 1.0, "masked": 0.0, "mix": 8},
        # a batch's step with the alternatives that an API returns, temperature 0.8
        {"name": "logprobs, a batch's step", "op": "logprobs", "n": 64, "vocab": 128256, "type": "f32", "k": 20, "m": 1, "scale": 1.25, "masked": 0.0, "mix": 9},
        # a corpus is scored in half precision, rows of an odd length (no row begins where the one before it did), some tokens forbidden
        {"name": "logprobs, scoring", "op": "logprobs", "n": 3001, "vocab": 100003, "type": "bf16", "k": 3, "m": 2, "scale": 1.0, "masked": 0.25, "mix": 10},
        # one conversation on the small model: its trees' masks, what the target accepts of them, the cache's rows moved together
        {"name": "accept, a small model", "op": "accept", "nseq": 2, "lo": 20, "hi": 300, "t": 8, "page": 16, "nkv": 3, "d": 64, "layers": 30, "mix": 11},
        # the same for a batch of 64 with 32 layers
        {"name": "accept, a batch", "op": "accept", "nseq": 64, "lo": 70, "hi": 1500, "t": 26, "page": 16, "nkv": 8, "d": 128, "layers": 32, "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    op = rng.choice(("tree", "tree", "tree", "sinks", "sinks", "sinks", "logprobs", "logprobs", "logprobs", "accept"))
    d, nkv, group = rng.choice(((64, 3, 3), (64, 1, 8), (80, 4, 1), (96, 4, 5), (128, 8, 4), (128, 4, 7), (128, 1, 16), (256, 2, 8), (256, 1, 4)))
    page, typ = rng.choice((16, 32, 64)), rng.choice(("f32", "f16", "bf16"))
    if op == "logprobs":
        n = _log(rng, 1, 4000)
        vocab = _log(rng, 100, max(200, min(200000, 250000000 // n)))
        return {"op": op, "n": n, "vocab": vocab, "type": typ, "k": rng.choice((0, 1, 5, 20, rng.randint(1, 64))), "m": rng.choice((0, 1, 1, 7)),
                "scale": rng.choice((1.0, 1.0, 0.7, 2.0)), "masked": rng.choice((0.0, 0.0, 0.5, 0.999)), "mix": mix}
    if op == "accept":
        t = rng.randint(1, 64)
        lo = t + _log(rng, 1, 300)
        return {"op": op, "nseq": _log(rng, 1, 64), "lo": lo, "hi": lo + _log(rng, 1, 1000), "t": t, "page": page, "nkv": nkv, "d": d, "layers": _log(rng, 1, 24), "mix": mix}
    nseq = _log(rng, 1, 64)
    if op == "tree":
        t = _log(rng, 2, 96)
        hi = t + _log(rng, 1, max(2, min(100000, 131072 // nseq)))
    else:
        t = rng.choice((1, 1, 1, 3, _log(rng, 4, max(8, 3000 // nseq))))
        hi = t + _log(rng, 1, max(2, min(120000, 131072 // nseq, 40000000 // (nseq * t * group))))
    window = _log(rng, 1, hi + 1)
    return {"op": "attn", "tree": op == "tree", "nseq": nseq, "lo": rng.choice((t, hi)), "hi": hi, "t": t, "nh": nkv * group, "nkv": nkv, "d": d, "page": page, "type": typ,
            "window": rng.choice((0, window)) if op == "tree" else window, "sinks": rng.choice((0, 1, 4, _log(rng, 1, 200))), "mix": mix}


# ---------------------------------------------------------------- sizes

def _padded(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def _block_bytes(page, d):
    dp = _padded(d)
    return 2 * page * (dp // 2 + dp // 16)


def _lengths(c):
    """The sequences' lengths, and how many of their last tokens are new."""
    r = random.Random(c["mix"])
    lens = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["nseq"] - 1)]
    if c["lo"] == 0 and c["nseq"] > 1:
        lens[1] = 0
    t = c["t"]
    news = [t] + [r.randint(max(1, t // 3), t) for _ in range(c["nseq"] - 1)]
    return lens, news


def _page_plan(c):
    """A pool's state as a serving process has it: the sequences' pages scattered over it, some of them free."""
    lens, _ = _lengths(c)
    page, r = c["page"], random.Random(c["mix"] + 1)
    need = [-(-n // page) for n in lens]
    npages = sum(need) + max(sum(need) // 8, 8)
    ids = list(range(npages))
    r.shuffle(ids)
    maxp = max(need) + 2
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n] + [-1] * (maxp - n))
        at += n
    return lens, tables, ids[at:], npages, maxp


def _trees(news, r):
    """Parents of drafted trees: token 0 the root, then level by level, each token's parent one of the level before."""
    trees = []
    for t in news:
        parents, level = [-1], [0]
        while len(parents) < t:
            width = min(t - len(parents), r.randint(1, max(2, t // 3)))
            ups = sorted(r.choice(level) for _ in range(width))
            level = list(range(len(parents), len(parents) + width))
            parents += ups
        trees.append(parents)
    return trees


def _drafts(news, seed):
    """Drafted trees with their tokens, and the target's tokens: at three of four tokens that have one, a child's.  A token on the accepted path is either in its
    place already or beyond every place that the path is moved to, so that a pass can be called on the same state again."""
    r = random.Random(seed)
    trees, tokens, targets = _trees(news, r), [], []
    for parents in trees:
        t = len(parents)
        ids = r.sample(range(49152), t)
        depth = [0] * t
        for j in range(1, t):
            depth[j] = depth[parents[j]] + 1
        want = [r.randrange(49152, 65536) for _ in range(t)]
        for j in r.sample(range(1, t), t - 1):
            if (j == depth[j] or j > max(depth)) and r.random() < 0.75:
                want[parents[j]] = ids[j]
        tokens.append(ids)
        targets.append(want)
    return trees, tokens, targets


def _path(parents, ids, want):
    """The accepted path of one tree."""
    path = [0]
    while True:
        nxt = [j for j in range(1, len(parents)) if parents[j] == path[-1] and ids[j] == want[path[-1]]]
        if not nxt:
            return path
        path.append(nxt[0])


def work(c):
    if c["op"] == "logprobs":
        es = 4 if c["type"] == "f32" else 2
        return {"bytes": c["n"] * (c["vocab"] * es + 8 * c["m"] + 8 + 8 * c["k"]), "flops": 6 * c["n"] * c["vocab"]}
    lens, news = _lengths(c)
    if c["op"] == "attn":
        es, dp = 4 if c["type"] == "f32" else 2, _padded(c["d"])
        keys = pairs = 0
        for n, t in zip(lens, news):
            base = n - t
            if c["window"]:
                first = max(0, base - c["window"] + 1)
                keys += n - first + min(first, c["sinks"])
            else:
                keys += n
            if c["tree"]:  # a path's length is small beside the context: its root and some drafts
                pairs += t * (min(base, c["window"] + c["sinks"]) if c["window"] else base) + 4 * t
            else:
                seen = np.maximum(base + np.arange(t) + 1, 0)
                pairs += int(np.minimum(seen, c["window"] + np.minimum(c["sinks"], np.maximum(seen - c["window"], 0))).sum()) if c["window"] else int(seen.sum())
        return {"bytes": 2 * keys * c["nkv"] * (dp // 2 + dp // 16) + sum(news) * c["nh"] * (2 * c["d"] * es + 4) + 4 * sum(-(-n // c["page"]) for n in lens)
                + (4 * sum(news) * -(-c["t"] // 32) if c["tree"] else 0), "flops": 4 * c["d"] * c["nh"] * pairs}
    trees, tokens, targets = _drafts(news, c["mix"])
    moved = sum(sum(1 for k, j in enumerate(_path(*x)) if j != k) for x in zip(trees, tokens, targets))
    dp = _padded(c["d"])
    row = 2 * c["nkv"] * (dp // 2 + dp // 16)
    return {"bytes": 2 * moved * c["layers"] * row + sum(news) * (3 * 4 + 4 * -(-c["t"] // 32) + 8) + 16 * c["nseq"] + 8 * sum(t // c["page"] + 2 for t in news), "flops": 0}


# ---------------------------------------------------------------- the stored form

_PLACES = {}


def _places(page, d, device):
    """Places of the codes in a block's code areas: two int64 [page, dp] of nibble numbers (nibble n is byte n // 2, the low half where n is even).

    A row is cut into planes of up to 128 elements.  Keys: the 16-byte quarter t of a plane's row holds elements 8t..8t+7 of each of its
    32-element groups.  Values: the eighth g holds elements 4g..4g+3 of each group, and every second pair of rows has its eighths exchanged in halves."""
    key = (page, _padded(d), str(device))
    if key not in _PLACES:
        dp = _padded(d)
        w = min(dp // 32, 4)
        r, i = torch.arange(page)[:, None], torch.arange(dp)[None, :]
        group = i // 32
        plane, g = group // 4, group % 4
        e = i % 32
        base = (plane * page + r) * 4 * w
        k = (base + (e // 8) * w + g) * 8 + e % 8
        chunk = (e // 4) ^ (4 * ((r >> 1) & 1))
        v = ((plane * page + r) * 8 * w + chunk * w + g) * 4 + e % 4
        _PLACES[key] = (k.to(device), v.to(device))
    return _PLACES[key]


def _parts(page, d):
    """Byte ranges of a block: keys' codes, keys' steps, values' codes, values' steps."""
    dp = _padded(d)
    c, s = page * dp // 2, page * dp // 16
    return (0, c), (c, c + s), (c + s, 2 * c + s), (2 * c + s, 2 * c + 2 * s)


def _quantize(x):
    """x f32 [..., dp] -> codes int32 [..., dp] and steps f16 [..., dp / 32]."""
    g = x.unflatten(-1, (-1, 32))
    hi, lo = g.amax(-1).clamp_min(0.0), g.amin(-1).clamp_max(0.0)
    step = (torch.where(hi >= -lo, hi, lo) * -0.125).to(torch.float16)
    s = step.float()[..., None]
    inv = torch.where(s == 0, torch.zeros_like(s), 1.0 / s)
    codes = (g * inv).round().clamp(-8, 7) + 8
    return codes.to(torch.int32).flatten(-2), step


def _pack(x, place):
    """x f32 [blocks, page, dp] -> (code bytes [blocks, page * dp / 2], step bytes [blocks, page * dp / 16]) as uint8."""
    codes, step = _quantize(x)
    n = codes.shape[0]
    nib = torch.empty((n, codes.shape[1] * codes.shape[2]), dtype=torch.uint8, device=x.device)
    nib[:, place.flatten()] = codes.flatten(1).to(torch.uint8)
    return nib[:, 0::2] | (nib[:, 1::2] << 4), step.flatten(1).contiguous().view(torch.uint8)


def _unpack(blocks, page, d):
    """blocks uint8 [n, block bytes] -> keys and values f32 [n, page, d]."""
    both = []
    parts = _parts(page, d)
    for (c0, c1), (s0, s1), place in zip(parts[0::2], parts[1::2], _places(page, d, blocks.device)):
        b = blocks[:, c0:c1]
        nib = torch.stack((b & 15, b >> 4), -1).flatten(1)
        codes = nib[:, place.flatten()].unflatten(1, (page, -1, 32))
        step = blocks[:, s0:s1].contiguous().view(torch.float16).unflatten(1, (page, -1, 1))
        both.append(((codes.float() - 8.0) * step.float()).flatten(-2)[..., :d])
    return both


# ---------------------------------------------------------------- the operators in plain form

def _bits(masks, t):
    """masks int32 [..., words] -> which of t drafts they mark."""
    return ((masks[..., None] >> torch.arange(32, device=masks.device)) & 1).flatten(-2)[..., :t] != 0


def _attn_plain(s, c):
    page, d, nkv, nseq, window, sinks = c["page"], c["d"], c["nkv"], c["nseq"], c["window"], c["sinks"]
    q, lens, start = s["q"], s["lens"].long(), s["q_start"].long()
    tables = s["tables"][:, : -(-c["hi"] // page)]
    blocks = s["pool"].unflatten(1, (nkv, -1))[tables.clamp_min(0).long()]
    k, v = (x.unflatten(0, (nseq, -1, nkv)).transpose(1, 2).flatten(2, 3) for x in _unpack(blocks.flatten(0, 2), page, d))
    key = torch.arange(k.shape[2], device=q.device)
    there = (key < lens[:, None])[:, None, :, None]
    k, v = torch.where(there, k, 0.0), torch.where(there, v, 0.0)
    t = torch.arange(c["t"], device=q.device)
    new = start[1:] - start[:-1]
    at = (start[:-1, None] + t).clamp_max(q.shape[0] - 1)
    base = (lens - new)[:, None, None]
    if c["tree"]:
        marked = _bits(s["masks"][at], c["t"]) & (t < new[:, None])[:, None, :]
        draft = (key - base).clamp(0, c["t"] - 1).expand(-1, c["t"], -1)
        seen = (key < lens[:, None, None]) & ((key < base) | marked.gather(-1, draft))
        if window:
            order = torch.cumsum(seen, -1)
            seen &= (order > order[..., -1:] - window) | (key < sinks)
    else:
        pos = base + t[:, None]
        seen = (key <= pos) & ((key > pos - window) | (key < sinks)) if window else key <= pos
    rows = q.float()[at].unflatten(2, (nkv, -1)).permute(0, 2, 1, 3, 4)
    scores = (rows.flatten(2, 3) @ k.transpose(-1, -2)).mul_(d ** -0.5).unflatten(2, (c["t"], -1))
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(top.clamp_min(-1e30)))
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (c["t"], -1)) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    valid = t < new[:, None]
    s["out"][at[valid]] = out.permute(0, 2, 1, 3, 4).flatten(2, 3)[valid].to(q.dtype)
    s["lse"][at[valid]] = lse.permute(0, 2, 1, 3).flatten(2, 3)[valid]
    return {"out": s["out"], "lse": s["lse"]}


def _logprobs_plain(s, c):
    x, got = s["logits"].float(), {}
    # values in their order as whole numbers, the lower index first where two are equal
    if c["k"]:
        b = (x + 0.0).view(torch.int32)
        order = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long() * (1 << 32) + ((1 << 31) - torch.arange(c["vocab"], device=x.device))
        got["top_tokens"] = torch.topk(order, c["k"], -1).indices.to(torch.int32)
        del order
    x = x * c["scale"]
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    z = x - lse
    got["entropy"] = -(torch.where(e > 0, e * z, 0.0).sum(-1) / total[:, 0])
    got["lse"] = lse[:, 0]
    if c["m"]:
        got["logprobs"] = z.gather(1, s["tokens"].long())
    if c["k"]:
        got["top_logprobs"] = z.gather(1, got["top_tokens"].long())
    return got


def _keep_plain(m, pool, c, rows, start, keep, nkeep):
    """The kept drafts' rows moved together behind the context in every layer, the lengths lowered, the pages past them given back."""
    page, d, nkv, dp = c["page"], c["d"], c["nkv"], _padded(c["d"])
    new = start[1:] - start[:-1]
    old = m["lens"][rows].long()
    base = old - new
    t = torch.arange(c["t"], device=rows.device)
    kept = t < nkeep[:, None]
    from_ = torch.where(kept, keep[(start[:-1, None] + t).clamp_max(keep.shape[0] - 1)].long(), 0)
    seq, k = torch.nonzero(kept & (from_ != t), as_tuple=True)
    bb = _block_bytes(page, d)
    flat = pool.view(torch.uint8).flatten(1)

    def bytes_of(place):
        pg, r = m["tables"][rows[seq], place // page].long(), place % page
        block = (pg[:, None] * nkv + torch.arange(nkv, device=rows.device)) * bb
        parts = []
        for (c0, _), (s0, _), nib in zip(_parts(page, d)[0::2], _parts(page, d)[1::2], _places(page, d, rows.device)):
            parts.append(c0 + nib[r, 0::2] // 2)
            parts.append(s0 + r[:, None] * (dp // 16) + torch.arange(dp // 16, device=rows.device))
        return (block[..., None] + torch.cat(parts, -1)[:, None]).flatten()

    flat[:, bytes_of(base[seq] + k)] = flat[:, bytes_of(base[seq] + from_[seq, k])]
    now = base + nkeep
    tables = m["tables"][rows]
    col = torch.arange(tables.shape[1], device=rows.device)
    gone = (col >= ((now + page - 1) // page)[:, None]) & (col < ((old + page - 1) // page)[:, None])
    npages = m["refs"].shape[0]
    before = m["refs"].clone()
    less = torch.zeros(npages + 1, dtype=torch.int32, device=rows.device)
    less.index_add_(0, torch.where(gone, tables.long(), npages).flatten(), torch.ones_like(tables).flatten())
    m["refs"] -= less[:npages]
    freed = (m["refs"] == 0) & (before > 0)
    place = torch.where(freed, m["nfree"] + torch.cumsum(freed, 0) - 1, npages)
    wide = torch.cat((m["free"], m["free"][:1]))
    wide[place] = torch.arange(npages, dtype=torch.int32, device=rows.device)
    m["free"].copy_(wide[:npages])
    m["nfree"] += freed.sum()
    m["lens"][rows] = now.to(torch.int32)
    m["tables"][rows] = torch.where(gone, -1, tables)


def _accept_plain(s, c):
    start, T = s["q_start"].long(), c["t"]
    new = start[1:] - start[:-1]
    t = torch.arange(T, device=start.device)
    at = (start[:-1, None] + t).clamp_max(s["parents"].shape[0] - 1)
    valid = t < new[:, None]
    parents = torch.where(valid, s["parents"][at].long(), -1)
    # a token's ancestors and itself: paths of any length through the parents
    up = (parents[..., None] == t).double()
    above = torch.linalg.matrix_power(up + torch.eye(T, device=up.device, dtype=up.dtype), T) > 0.5
    words = s["masks"].shape[1]
    bits = (torch.nn.functional.pad(above, (0, 32 * words - T)).unflatten(-1, (words, 32)).long() << torch.arange(32, device=up.device)).sum(-1)
    s["masks"][at[valid]] = ((bits + (1 << 31)) % (1 << 32) - (1 << 31)).to(torch.int32)[valid]
    s["depth"][at[valid]] = (above.sum(-1) - 1).to(torch.int32)[valid]
    # the path: tokens that the target chose after their parent, the first such child of it, all ancestors likewise
    ids, want = s["draft"][at], s["target"][at]
    chosen = (parents >= 0) & valid & (ids == want.gather(1, parents.clamp_min(0)))
    twin = (parents[:, :, None] == parents[:, None, :]) & chosen[:, :, None] & chosen[:, None, :] & (t < t[:, None])
    good = (chosen & ~twin.any(-1)) | (t == 0)
    path = valid & ~(above & ~good[:, None, :]).any(-1)
    keep = torch.where(path, t, T).sort(-1).values
    s["keep"][at[valid]] = torch.where(keep < T, keep, -1).to(torch.int32)[valid]
    nkeep = path.sum(-1)
    s["nkeep"].copy_(nkeep)
    s["next"].copy_(want.gather(1, torch.where(path, t, 0).amax(-1, keepdim=True))[:, 0])
    s["state"].copy_(s["saved"])
    _keep_plain(s["meta"], s["pool"], c, s["rows"].long(), start, s["keep"], nkeep)
    s["status"].zero_()
    return {n: s[n] for n in ("masks", "depth", "keep", "nkeep", "next", "status", "state", "pool")}


# ---------------------------------------------------------------- what a pass has in hand

def _fill(pool, c, gen):
    """Random keys (with an offset of each channel's own) and values, quantized into every block of the pool [blocks, block bytes], a part at a time."""
    page, d, dp = c["page"], c["d"], _padded(c["d"])
    place, parts = _places(page, d, pool.device), _parts(page, d)
    shift = torch.randn(dp, device=pool.device, generator=gen)
    step = max(1, (1 << 26) // (page * dp))
    for b in range(0, pool.shape[0], step):
        n = min(step, pool.shape[0] - b)
        for k in (0, 1):
            x = torch.randn((n, page, dp), device=pool.device, generator=gen)
            if k == 0:
                x += shift
            x[..., d:] = 0.0
            code, st = _pack(x, place[k])
            pool[b:b + n, parts[2 * k][0]:parts[2 * k][1]] = code
            pool[b:b + n, parts[2 * k + 1][0]:parts[2 * k + 1][1]] = st


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + c["mix"])
    s = {"case": c}
    if c["op"] == "logprobs":
        x = torch.randn((c["n"], c["vocab"]), device=dev, generator=gen) * 2.5
        # a few likely tokens in each row
        likely = torch.randint(0, c["vocab"], (c["n"], 6), device=dev, generator=gen)
        x.scatter_add_(1, likely, torch.rand((c["n"], 6), device=dev, generator=gen) * 12)
        tokens = torch.cat((likely[:, :1], torch.randint(0, c["vocab"], (c["n"], 8), device=dev, generator=gen)), 1)[:, :c["m"]]
        if c["masked"]:
            x.masked_fill_(torch.rand(c["vocab"], device=dev, generator=gen) < c["masked"], -math.inf)
            x[:, 17] = 1.0  # no row is left without a token
        s["logits"], s["tokens"] = x.to(_TYPES[c["type"]]), tokens.to(torch.int32).contiguous()
        f32 = dict(dtype=torch.float32, device=dev)
        s["out"] = {"entropy": torch.empty(c["n"], **f32), "lse": torch.empty(c["n"], **f32)}
        if c["m"]:
            s["out"]["logprobs"] = torch.empty((c["n"], c["m"]), **f32)
        if c["k"]:
            s["out"]["top_tokens"] = torch.empty((c["n"], c["k"]), dtype=torch.int32, device=dev)
            s["out"]["top_logprobs"] = torch.empty((c["n"], c["k"]), **f32)
        return s
    lens, tables, free, npages, maxp = _page_plan(c)
    _, news = _lengths(c)
    bb, n, words = _block_bytes(c["page"], c["d"]), sum(news), -(-c["t"] // 32)
    s["q_start"] = _ints([sum(news[:i]) for i in range(c["nseq"] + 1)])
    if c["op"] == "attn":
        s["pool"] = torch.empty((npages, c["nkv"] * bb), dtype=torch.uint8, device=dev)
        _fill(s["pool"].view(-1, bb), c, gen)
        s["tables"], s["lens"] = _ints(tables), _ints(lens)
        s["q"] = torch.randn((n, c["nh"], c["d"]), device=dev, generator=gen).to(_TYPES[c["type"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, c["nh"]), dtype=torch.float32, device=dev)
        if c["tree"]:
            masks = []
            for parents in _trees(news, random.Random(seed * 1000003 + c["mix"])):
                m = []
                for j, p in enumerate(parents):
                    m.append((m[p] if p >= 0 else 0) | 1 << j)
                masks += [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in m]
            s["masks"] = torch.from_numpy(np.array(masks, dtype=np.uint32).view(np.int32)).to(dev)
        return s
    s["pool"] = torch.randint(-2**31, 2**31 - 1, (c["layers"], npages, c["nkv"] * bb // 4), dtype=torch.int32, device=dev, generator=gen)
    refs = [0] * npages
    for x in (x for t in tables for x in t if x >= 0):
        refs[x] += 1
    # one buffer for the pool's whole state, so that one copy brings it back before every pass
    s["saved"] = _ints([len(free)] + free + [-1] * (npages - len(free)) + refs + lens + [x for t in tables for x in t])
    s["state"] = s["saved"].clone()
    s["meta"] = dict(zip(("nfree", "free", "refs", "lens", "tables"), s["state"].split([1, npages, npages, c["nseq"], c["nseq"] * maxp])))
    s["meta"]["tables"] = s["meta"]["tables"].view(c["nseq"], maxp)
    for name, x in zip(("parents", "draft", "target"), _drafts(news, seed * 1000003 + c["mix"])):
        s[name] = _ints([y for z in x for y in z])
    s["rows"] = _ints(list(range(c["nseq"])))
    i32 = dict(dtype=torch.int32, device=dev)
    s["masks"], s["depth"], s["keep"] = torch.zeros((n, words), **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
    s["nkeep"], s["next"], s["status"] = (torch.zeros(c["nseq"], **i32) for _ in range(3))
    return s


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "attn":
        return _attn_plain(s, c)
    return _logprobs_plain(s, c) if c["op"] == "logprobs" else _accept_plain(s, c)


def _run_own(s, c):
    import block_quantized_weight_quantize_gb300 as qb
    if c["op"] == "logprobs":
        o = s["out"]
        qb.q_logprobs(s["logits"], tokens=s["tokens"] if c["m"] else None, scale=c["scale"], logprobs=o.get("logprobs"), entropy=o["entropy"], lse=o["lse"],
                      top_tokens=o.get("top_tokens"), top_logprobs=o.get("top_logprobs"))
        return o
    h = s.get("held")
    if h is None:  # what a serving process makes once: the handles of its cache, its sequences and pages, and its workspace
        h = s["held"] = {}
        if c["op"] == "attn":
            h["cache"] = qb.Kv4(s["pool"], c["page"], c["nkv"], c["d"])
            h["seqs"] = qb.KvSeqs(s["tables"], s["lens"], q_start=s["q_start"])
            h["ws"] = torch.empty(qb.kv4_attn_workspace_bytes(h["cache"], s["q"], h["seqs"]), dtype=torch.uint8, device="cuda")
        else:
            m = s["meta"]
            h["pages"] = qb.KvPages(c["page"], m["nfree"], m["free"], m["refs"], m["lens"], m["tables"])
    if c["op"] == "accept":
        qb.kv_tree_masks(s["parents"], s["masks"], s["depth"], q_start=s["q_start"])
        qb.kv_tree_accept(s["parents"], s["draft"], s["target"], s["keep"], s["nkeep"], s["next"], q_start=s["q_start"])
        s["state"].copy_(s["saved"])
        qb.kv4_keep(h["pages"], s["pool"], c["nkv"], c["d"], s["rows"], s["q_start"], s["keep"], s["nkeep"], s["status"])
        return {n: s[n] for n in ("masks", "depth", "keep", "nkeep", "next", "status", "state", "pool")}
    if c["tree"]:
        qb.kv4_attn_tree(h["cache"], s["q"], h["seqs"], s["masks"], c["d"] ** -0.5, s["out"], lse=s["lse"], window=c["window"], sinks=c["sinks"], workspace=h["ws"])
    else:
        qb.kv4_attn_sinks(h["cache"], s["q"], h["seqs"], c["d"] ** -0.5, s["out"], c["window"], c["sinks"], lse=s["lse"], workspace=h["ws"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_logprobs(s, c):
    got = {n: [] for n in s["out"]}
    for i in range(0, c["n"], max(1, (1 << 26) // c["vocab"])):
        x = s["logits"][i:i + max(1, (1 << 26) // c["vocab"])].double()
        z = x * c["scale"]
        lse = torch.logsumexp(z, -1, keepdim=True)
        logp = z - lse
        p = torch.exp(logp)
        got["lse"].append(lse[:, 0])
        got["entropy"].append(torch.where(p > 0, -p * logp, 0.0).sum(-1))
        if c["m"]:
            got["logprobs"].append(torch.gather(logp, 1, s["tokens"][i:i + x.shape[0]].long()))
        if c["k"]:
            got["top_logprobs"].append(logp.sort(-1, descending=True).values[:, :c["k"]])
    return {n: torch.cat(x) if x else None for n, x in got.items()}


def exact(case, seed):
    """attn: softmax(q k' / sqrt(d)) v over the keys that a token sees, each token's set of them built by itself, the elements taken from the cache one byte at a
    time.  logprobs: log softmax of the scaled logits, its entropy, its largest values.  accept: whole numbers, which have to be equal."""
    c = case
    if c["op"] == "accept" or (c["op"] == "logprobs" and c["n"] * c["vocab"] > 2e9):
        return None
    s = prepare(case, seed)
    if c["op"] == "logprobs":
        return _exact_logprobs(s, c)
    dp, page, nkv, d = _padded(c["d"]), c["page"], c["nkv"], c["d"]
    lens, news = _lengths(c)
    if max(lens) * nkv * dp * 32 > 100e9 or max(n * t for n, t in zip(lens, news)) * c["nh"] * 24 > 100e9:
        return None
    w, bb = min(dp // 32, 4), _block_bytes(page, d)
    i = torch.arange(d, device="cuda")
    plane, g, e = i // 128, i // 32 % 4, i % 32
    code_bytes, step_bytes = page * dp // 2, page * dp // 16
    flat = s["pool"].reshape(-1)
    out, lse, at = [], [], 0
    for b, (n, t) in enumerate(zip(lens, news)):
        q = s["q"][at:at + t].double().reshape(t, nkv, -1, d)
        seen = np.zeros((t, n), dtype=bool)
        marks = s["masks"][at:at + t].cpu().numpy().view(np.uint32) if c["tree"] else None
        for j in range(t):
            if c["tree"]:
                drafts = [n - t + x for x in range(t) if n - t + x >= 0 and marks[j, x // 32] >> (x % 32) & 1]
                keys = np.concatenate((np.arange(max(0, n - t)), np.array(drafts, dtype=np.int64)))
            else:
                keys = np.arange(max(0, n - t + j + 1))
            if c["window"]:
                keys = np.union1d(keys[-c["window"]:], keys[keys < c["sinks"]])
            seen[j, keys.astype(np.int64)] = True
        at += t
        seen = torch.from_numpy(seen).to("cuda")
        key = torch.arange(n, device="cuda")
        r = (key % page)[:, None]
        base = s["tables"][b].long()[key // page][:, None] * nkv * bb
        sides = []
        for side in (0, 1):
            area = side * (code_bytes + step_bytes)
            row = area + (plane * page + r) * 16 * w
            if side == 0:
                byte, odd = row + e // 8 * 4 * w + g * 4 + e % 8 // 2, e % 2
            else:
                byte, odd = row + (e // 4 ^ 4 * (r // 2 % 2)) * 2 * w + g * 2 + e % 4 // 2, e % 2
            heads = []
            for h in range(nkv):
                o = base + h * bb
                code = (flat[o + byte].int() >> (4 * odd)) & 15
                lo = o + area + code_bytes + r * (dp // 16) + i // 32 * 2
                bits = flat[lo].int() | flat[lo + 1].int() << 8
                heads.append((code - 8).double() * bits.to(torch.int16).view(torch.float16).double())
            sides.append(torch.stack(heads))
        k, v = sides
        z = torch.einsum("thgd,hnd->thgn", q, k) / math.sqrt(d)
        z = torch.where(seen[:, None, None, :], z, -math.inf)
        total = torch.logsumexp(z, -1) if n else z.new_full((t, nkv, c["nh"] // nkv), -math.inf)
        p = torch.where(torch.isfinite(total)[..., None], torch.exp(z - total[..., None]), 0.0)
        out.append(torch.einsum("thgn,hnd->thgd", p, v).reshape(t, -1, d))
        lse.append(total.reshape(t, -1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
