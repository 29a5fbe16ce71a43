"""The paged 4-bit key/value cache: what its operators compute, in plain torch, and the cases they are timed on.

The cache holds, per page and key head, one block of bytes: the keys' codes, the keys' steps, the values' codes, the
values' steps.  A row (one token, one head) of d elements is stored as dp (d rounded up to 64, 128 or 256, the rest
zeros) 4-bit codes with one f16 step per 32 of them; an element is (code - 8) * step.  `_places` below gives the place
of every code.  The operators: `kv4_append` (rows into the cache), `kv4_read` (rows out of it), `kv4_attn` (causal
attention of new tokens over the cache), and the pages' own: `kv_pages_extend`, `kv_pages_fork`, `kv_pages_free`,
`kv_pages_compact`, `kv_pages_copy`.
"""
import math
import random

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decoding step's new keys and values of a batch of 64 (8B-class heads): the smallest call, latency counts
        {"name": "append, a step", "op": "append", "n": 64, "nkv": 8, "d": 128, "page": 16, "type": "f32", "mix": 1},
        # a batch of prompts written at once, from a half-precision model
        {"name": "append, prompts", "op": "append", "n": 20011, "nkv": 8, "d": 128, "page": 64, "type": "bf16", "mix": 2},
        # a chat's first tokens on a small model with 9 query and 3 key heads: latency
        {"name": "attention, one short sequence", "op": "attn", "nseq": 1, "lo": 37, "hi": 37, "t": 1, "nh": 9, "nkv": 3, "d": 64,
         "page": 16, "type": "f32", "window": 0, "mix": 3},
        # the ordinary serving step: 64 sequences of unequal length, one of them still empty
        {"name": "attention, a batch's step", "op": "attn", "nseq": 64, "lo": 0, "hi": 8192, "t": 1, "nh": 32, "nkv": 8, "d": 128,
         "page": 16, "type": "f32", "window": 0, "mix": 4},
        # one long document: the key axis has to be split
        {"name": "attention, one long sequence", "op": "attn", "nseq": 1, "lo": 131071, "hi": 131071, "t": 1, "nh": 32, "nkv": 8, "d": 128,
         "page": 64, "type": "bf16", "window": 0, "mix": 5},
        # wide heads shared eight ways, with a sliding window
        {"name": "attention, wide heads, window", "op": "attn", "nseq": 48, "lo": 100, "hi": 5000, "t": 1, "nh": 16, "nkv": 2, "d": 256,
         "page": 32, "type": "f16", "window": 2048, "mix": 6},
        # several drafted tokens a sequence checked at once
        {"name": "attention, drafted tokens", "op": "attn", "nseq": 24, "lo": 1, "hi": 4097, "t": 5, "nh": 32, "nkv": 8, "d": 128,
         "page": 16, "type": "f32", "window": 0, "mix": 7},
        # a prompt's chunk over what is cached already
        {"name": "attention, a prompt's chunk", "op": "attn", "nseq": 1, "lo": 8192, "hi": 8192, "t": 2048, "nh": 32, "nkv": 8, "d": 128,
         "page": 64, "type": "bf16", "window": 0, "mix": 8},
        # a few short prompts of unequal length, in f32, on the small model
        {"name": "attention, short prompts", "op": "attn", "nseq": 5, "lo": 90, "hi": 1500, "t": 700, "nh": 9, "nkv": 3, "d": 64,
         "page": 16, "type": "f32", "window": 0, "mix": 9},
        # one conversation branches: two sequences end, two are forked from others, each goes on by a token
        {"name": "pages, a small fork", "op": "fork", "nseq": 8, "n": 2, "lo": 20, "hi": 300, "page": 16, "nkv": 3, "d": 64, "layers": 30, "mix": 10},
        # a beam step: 24 of 64 beams end, as many are forked from others
        {"name": "pages, a beam step", "op": "fork", "nseq": 64, "n": 24, "lo": 100, "hi": 2000, "page": 64, "nkv": 8, "d": 128, "layers": 32, "mix": 11},
        # half the sequences end and the pool is moved together, to give its end back
        {"name": "pages, compacting", "op": "compact", "nseq": 32, "n": 16, "lo": 30, "hi": 1400, "page": 16, "nkv": 8, "d": 128, "layers": 32, "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    mix = rng.randrange(1 << 30)
    d, nkv, group = rng.choice(((64, 3, 3), (64, 1, 8), (80, 4, 1), (96, 4, 5), (128, 8, 4), (128, 4, 7), (128, 1, 16), (256, 2, 8), (256, 1, 4)))
    page, typ = rng.choice((16, 32, 64)), rng.choice(("f32", "f16", "bf16"))
    op = rng.choice(("append", "attn", "attn", "attn", "attn", "prompt", "prompt", "fork", "compact"))
    if op == "append":
        return {"op": op, "n": _log(rng, 1, 20000), "nkv": nkv, "d": d, "page": page, "type": typ, "mix": mix}
    if op == "attn":
        nseq = _log(rng, 1, 96)
        hi = _log(rng, 1, max(2, min(131071, 262144 // nseq)))
        return {"op": "attn", "nseq": nseq, "lo": rng.choice((0, 1, hi)), "hi": hi, "t": rng.choice((1, 1, 1, 2, 4, 7)), "nh": nkv * group, "nkv": nkv,
                "d": d, "page": page, "type": typ, "window": rng.choice((0, 0, 0, _log(rng, 1, hi + 1))), "mix": mix}
    if op == "prompt":
        nseq = rng.choice((1, 1, 2, 3, 5))
        hi = _log(rng, 40, 4000 // nseq)
        return {"op": "attn", "nseq": nseq, "lo": max(1, hi // 3), "hi": hi, "t": _log(rng, 20, max(21, min(hi, 1500))), "nh": nkv * group, "nkv": nkv,
                "d": d, "page": page, "type": typ, "window": rng.choice((0, 0, 0, _log(rng, 16, hi + 1))), "mix": mix}
    nseq = _log(rng, 2, 48)
    lo = _log(rng, 1, 200)
    return {"op": op, "nseq": nseq, "n": rng.randint(1, max(1, nseq // 2)), "lo": lo, "hi": lo + _log(rng, 1, 1000), "page": page, "nkv": nkv, "d": d,
            "layers": _log(rng, 1, 16), "mix": mix}


# ---------------------------------------------------------------- sizes

def _padded(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def _block_bytes(page, d):
    dp = _padded(d)
    return 2 * page * (dp // 2 + dp // 16)


def _lengths(c):
    """The sequences' lengths, and how many of their last tokens are new (for attention)."""
    r = random.Random(c["mix"])
    lens = [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["nseq"] - 1)]
    if c["lo"] == 0 and c["nseq"] > 1:
        lens[1] = 0
    t = c.get("t", 1)
    news = [t] + [r.randint(max(1, t // 3), t) for _ in range(c["nseq"] - 1)]
    return lens, news


def _page_plan(c):
    """A pool's state as a serving process has it: the sequences' pages scattered over it, some of them free."""
    lens, _ = _lengths(c)
    page, r = c["page"], random.Random(c["mix"] + 1)
    need = [-(-n // page) for n in lens]
    spare = max(4 * c.get("n", 0), sum(need) // 8, 8)
    npages = sum(need) + spare
    ids = list(range(npages))
    r.shuffle(ids)
    maxp = max(need) + 2
    tables, at = [], 0
    for n in need:
        tables.append(ids[at:at + n] + [-1] * (maxp - n))
        at += n
    return lens, tables, ids[at:], npages, maxp


def _fork_plan(c):
    """Which sequences end, and which ones the freed rows are forked from."""
    r = random.Random(c["mix"] + 2)
    rows = list(range(c["nseq"]))
    r.shuffle(rows)
    n = c["n"]
    ended, kept = rows[:n], rows[n:]
    return ended, [r.choice(kept) for _ in range(n)] if c["op"] == "fork" else [], kept


def work(c):
    if c["op"] == "append":
        rows, es = c["n"] * c["nkv"], 4 if c["type"] == "f32" else 2
        dp = _padded(c["d"])
        stored = dp // 2 + dp // 16
        return {"bytes": 2 * rows * (2 * c["d"] * es + 2 * stored) + 4 * c["n"], "flops": 2 * rows * c["d"] * 4}
    if c["op"] == "attn":
        lens, news = _lengths(c)
        es, dp = 4 if c["type"] == "f32" else 2, _padded(c["d"])
        keys = pairs = 0
        for n, t in zip(lens, news):
            first = max(0, n - t - c["window"] + 1) if c["window"] else 0
            keys += max(0, n - first)
            for j in range(t):
                pos = n - t + j
                pairs += max(0, min(pos + 1, c["window"] or pos + 1))
        return {"bytes": 2 * keys * c["nkv"] * (dp // 2 + dp // 16) + sum(news) * c["nh"] * (2 * c["d"] * es + 4) + 4 * sum(-(-n // c["page"]) for n in lens),
                "flops": 4 * c["d"] * c["nh"] * pairs}
    lens, tables, free, npages, maxp = _page_plan(c)
    ended, parents, kept = _fork_plan(c)
    page_bytes = c["nkv"] * _block_bytes(c["page"], c["d"])
    if c["op"] == "fork":
        moved = sum(1 for p in parents if lens[p] % c["page"])
    else:
        used = sorted(x for s in kept for x in tables[s] if x >= 0)
        moved = sum(1 for x in used if x >= len(used))
    ints = 1 + 2 * npages + c["nseq"] * (1 + maxp)
    return {"bytes": 2 * moved * c["layers"] * page_bytes + 2 * 4 * ints, "flops": 0}


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


def _row_bytes(slots, c):
    """For each row slot: its page, and the byte places in the block [n, dp / 2] and the elements [n, dp / 2, 2] that they hold, for keys and for values;
    a slot below zero has the place past the pool's end."""
    page, d = c["page"], c["d"]
    at = slots.clamp_min(0).long()
    out = []
    for (c0, _), place in zip(_parts(page, d)[0::2], _places(page, d, slots.device)):
        nib, element = place.sort(-1)
        out.append(((c0 + nib[:, 0::2] // 2)[at % page], element.unflatten(-1, (-1, 2))[at % page]))
    return at // page, at % page, out


# ---------------------------------------------------------------- the operators in plain form

def _append_plain(s, c):
    page, d, nkv, dp = c["page"], c["d"], c["nkv"], _padded(c["d"])
    pool = s["pool"].reshape(-1)
    bb = _block_bytes(page, d)
    pages, row, places = _row_bytes(s["slots"], c)
    block = (pages[:, None] * nkv + torch.arange(nkv, device=pool.device)) * bb
    got = {}
    for name, (at, element), (s0, _) in zip("kv", places, _parts(page, d)[1::2]):
        x = torch.nn.functional.pad(s[name].float(), (0, dp - d))
        codes, step = _quantize(x)
        pairs = codes.gather(-1, element.flatten(1)[:, None].expand(-1, nkv, -1)).unflatten(-1, (-1, 2))
        pool[(block[..., None] + at[:, None])] = (pairs[..., 0] | (pairs[..., 1] << 4)).to(torch.uint8)
        ng2 = dp // 16
        steps_at = block[..., None] + s0 + row[:, None, None] * ng2 + torch.arange(ng2, device=pool.device)
        pool[steps_at] = step.contiguous().view(torch.uint8)
        # read back
        b = pool[(block[..., None] + at[:, None])].int()
        back = torch.empty_like(codes)
        back.scatter_(-1, element.flatten(1)[:, None].expand(-1, nkv, -1), torch.stack((b & 15, b >> 4), -1).flatten(-2))
        st = pool[steps_at].view(torch.float16).float()[..., None]
        got[name] = ((back.unflatten(-1, (-1, 32)).float() - 8.0) * st).flatten(-2)[..., :d].to(s[name].dtype)
    return got


def _attn_plain(s, c):
    page, d, nkv, nh, nseq, window = c["page"], c["d"], c["nkv"], c["nh"], c["nseq"], c["window"]
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
    rows = q.float()[at].unflatten(2, (nkv, -1)).permute(0, 2, 1, 3, 4)
    scores = (rows.flatten(2, 3) @ k.transpose(-1, -2)).mul_(c["d"] ** -0.5).unflatten(2, (c["t"], -1))
    pos = (lens - new)[:, None] + t
    seen = key <= pos[..., None]
    if window:
        seen &= key > pos[..., None] - window
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(top.clamp_min(-1e30)))
    total = p.sum(-1, keepdim=True)
    out = (p.flatten(2, 3) @ v).unflatten(2, (c["t"], -1)) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    valid = t < new[:, None]
    out = out.permute(0, 2, 1, 3, 4).flatten(2, 3)
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)
    s["out"][at[valid]] = out[valid].to(q.dtype)
    s["lse"][at[valid]] = lse[valid]
    return {"out": s["out"], "lse": s["lse"]}


def _free_plain(m, rows, page):
    tables = m["tables"][rows]
    listed_ = torch.arange(tables.shape[1], device=rows.device) < ((m["lens"][rows].long() + page - 1) // page)[:, None]
    before = m["refs"].clone()
    npages = before.shape[0]
    less = torch.zeros(npages + 1, dtype=torch.int32, device=rows.device)
    less.index_add_(0, torch.where(listed_, tables.long(), npages).flatten(), torch.ones_like(tables).flatten())
    m["refs"] -= less[:npages]
    freed = (m["refs"] == 0) & (before > 0)
    place = torch.where(freed, m["nfree"] + torch.cumsum(freed, 0) - 1, npages)
    wide = torch.cat((m["free"], m["free"][:1]))
    wide[place] = torch.arange(npages, dtype=torch.int32, device=rows.device)
    m["free"].copy_(wide[:npages])
    m["nfree"] += freed.sum()
    m["lens"][rows] = 0
    m["tables"][rows] = -1


def _fork_plain(m, pool, parents, children, page):
    lens = m["lens"][parents].long()
    tail = lens % page != 0
    rank = torch.cumsum(tail, 0) - tail.long()
    fits = ~tail | (rank < m["nfree"])
    top = m["free"][(m["nfree"] - 1 - rank).clamp_min(0)].long()
    rows = m["tables"][parents].clone()
    last = (lens // page)[:, None]
    col = torch.arange(rows.shape[1], device=rows.device)
    shared = (col < last) & fits[:, None]
    old = rows.gather(1, last.clamp_max(rows.shape[1] - 1))[:, 0].long()
    rows = torch.where((col == last) & tail[:, None], top[:, None].to(rows.dtype), rows)
    m["tables"][children] = torch.where(fits[:, None], rows, m["tables"][children])
    m["lens"][children] = torch.where(fits, lens.to(torch.int32), m["lens"][children])
    npages = m["refs"].shape[0]
    more = torch.zeros(npages + 1, dtype=torch.int32, device=rows.device)
    more.index_add_(0, torch.where(shared, rows.long(), npages).flatten(), torch.ones_like(rows).flatten())
    taken = tail & fits
    more.index_add_(0, torch.where(taken, top, npages), torch.ones_like(lens, dtype=torch.int32))
    m["refs"] += more[:npages]
    m["nfree"] -= taken.sum()
    pool[:, top[taken]] = pool[:, old[taken]]
    return torch.where(fits, 0, -8).to(torch.int32)


def _extend_plain(m, rows, page):
    """One token more for each sequence in `rows`: the tokens' slots, and what became of each request."""
    old = m["lens"][rows].long()
    room = old < m["tables"].shape[1] * page
    need = (old % page == 0) & room
    rank = torch.cumsum(need, 0) - need.long()
    fits = room & (~need | (rank < m["nfree"]))
    top = m["free"][(m["nfree"] - 1 - rank).clamp_min(0)]
    col = (old // page).clamp_max(m["tables"].shape[1] - 1)
    entry = torch.where(need & fits, top, m["tables"][rows, col])
    m["tables"][rows, col] = entry
    npages = m["refs"].shape[0]
    wide = torch.cat((m["refs"], m["refs"][:1]))
    wide[torch.where(need & fits, top.long(), npages)] = 1
    m["refs"].copy_(wide[:npages])
    m["nfree"] -= (need & fits).sum()
    m["lens"][rows] = (old + fits).to(torch.int32)
    return torch.where(fits, entry * page + (old % page).to(torch.int32), -1), torch.where(fits, 0, -8).to(torch.int32)


def _compact_plain(m, pool, page):
    npages = m["refs"].shape[0]
    ids = torch.arange(npages, device=pool.device)
    held = m["refs"] > 0
    used = held.sum()
    moves, holes = held & (ids >= used), ~held & (ids < used)
    moves_rank, holes_rank = torch.cumsum(moves, 0) - 1, torch.cumsum(holes, 0) - 1
    to = torch.full((npages + 1,), 0, dtype=torch.int64, device=pool.device)
    to[torch.where(holes, holes_rank, npages)] = ids
    new = torch.where(moves, to[moves_rank.clamp_min(0)], ids)
    src, dst = ids[moves], new[moves]
    pool[:, dst] = pool[:, src]
    refs = torch.zeros_like(m["refs"])
    refs[:] = torch.where(ids < used, torch.where(held, m["refs"], 0), 0)
    refs[dst] = m["refs"][src]
    m["refs"].copy_(refs)
    m["tables"].copy_(torch.where(m["tables"] >= 0, new[m["tables"].clamp_min(0).long()].to(torch.int32), m["tables"]))
    free = npages - 1 - ids
    m["free"].copy_(torch.where(ids < npages - used, free, m["free"].long()).to(torch.int32))
    m["nfree"].copy_((npages - used).to(torch.int32))


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


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed * 1000003 + c["mix"])
    bb = _block_bytes(c["page"], c["d"])
    s = {"case": c}
    if c["op"] == "append":
        npages = -(-c["n"] // c["page"]) * 2 + 3
        s["pool"] = torch.zeros((npages, c["nkv"] * bb), dtype=torch.uint8, device=dev)
        typ = _TYPES[c["type"]]
        shift = torch.randn(c["d"], device=dev, generator=gen)
        s["k"] = (torch.randn((c["n"], c["nkv"], c["d"]), device=dev, generator=gen) + shift).to(typ)
        s["v"] = torch.randn((c["n"], c["nkv"], c["d"]), device=dev, generator=gen).to(typ)
        # runs of a page's rows on scattered pages, as the tokens of a batch lie
        pages = torch.randperm(npages, device=dev, generator=gen)[: -(-c["n"] // c["page"]) + 1]
        at = torch.arange(c["n"], device=dev) + c["mix"] % c["page"]
        s["slots"] = (pages[at // c["page"]] * c["page"] + at % c["page"]).to(torch.int32)
        s["k_back"], s["v_back"] = torch.empty_like(s["k"]), torch.empty_like(s["v"])
    elif c["op"] == "attn":
        lens, tables, _, npages, maxp = _page_plan(c)
        _, news = _lengths(c)
        s["pool"] = torch.empty((npages, c["nkv"] * bb), dtype=torch.uint8, device=dev)
        _fill(s["pool"].view(-1, bb), c, gen)
        s["tables"] = torch.tensor(tables, dtype=torch.int32, device=dev)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["q_start"] = torch.tensor([sum(news[:i]) for i in range(c["nseq"] + 1)], dtype=torch.int32, device=dev)
        n = sum(news)
        s["q"] = torch.randn((n, c["nh"], c["d"]), device=dev, generator=gen).to(_TYPES[c["type"]])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((n, c["nh"]), dtype=torch.float32, device=dev)
    else:
        lens, tables, free, npages, maxp = _page_plan(c)
        ended, parents, kept = _fork_plan(c)
        s["pool"] = torch.randint(-2**31, 2**31 - 1, (c["layers"], npages, c["nkv"] * bb // 4), dtype=torch.int32, device=dev, generator=gen)
        refs = [0] * npages
        for t in tables:
            for x in t:
                if x >= 0:
                    refs[x] += 1
        # one buffer for the pool's whole state, so that one copy brings it back before every pass
        flat = [len(free)] + free + [-1] * (npages - len(free)) + refs + lens + [x for t in tables for x in t]
        s["saved"] = torch.tensor(flat, dtype=torch.int32, device=dev)
        s["state"] = s["saved"].clone()
        s["meta"] = dict(zip(("nfree", "free", "refs", "lens", "tables"), s["state"].split([1, npages, npages, c["nseq"], c["nseq"] * maxp])))
        s["meta"]["tables"] = s["meta"]["tables"].view(c["nseq"], maxp)
        s["ended"] = torch.tensor(ended, dtype=torch.int32, device=dev)
        s["parents"] = torch.tensor(parents, dtype=torch.int32, device=dev)
        s["all"] = torch.arange(c["nseq"], dtype=torch.int32, device=dev)
        s["ones"] = torch.ones(c["nseq"], dtype=torch.int32, device=dev)
        s["slots"] = torch.empty(c["nseq"], dtype=torch.int32, device=dev)
        s["status"] = torch.empty(c["nseq"], dtype=torch.int32, device=dev)
        s["forked"] = torch.empty(c["n"], dtype=torch.int32, device=dev)
    return s


def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "append":
        return _append_plain(s, c)
    if c["op"] == "attn":
        return _attn_plain(s, c)
    m, pool, page = s["meta"], s["pool"], c["page"]
    s["state"].copy_(s["saved"])
    _free_plain(m, s["ended"].long(), page)
    if c["op"] == "compact":
        _compact_plain(m, pool, page)
        return {"state": s["state"], "pool": pool}
    s["forked"].copy_(_fork_plain(m, pool, s["parents"].long(), s["ended"].long(), page))
    slots, status = _extend_plain(m, s["all"].long(), page)
    s["slots"].copy_(slots)
    s["status"].copy_(status)
    return {"state": s["state"], "pool": pool, "slots": s["slots"], "status": s["status"], "forked": s["forked"]}


def _run_own(s, c):
    import block_quantized_weight_quantize_gb300 as qb
    h = s.get("held")
    if h is None:  # what a serving process makes once: the handles of its cache and its workspace
        h = s["held"] = {}
        if c["op"] in ("append", "attn"):
            h["cache"] = qb.Kv4(s["pool"], c["page"], c["nkv"], c["d"])
        if c["op"] == "attn":
            h["seqs"] = qb.KvSeqs(s["tables"], s["lens"], q_start=s["q_start"])
            h["ws"] = torch.empty(qb.kv4_attn_workspace_bytes(h["cache"], s["q"], h["seqs"]), dtype=torch.uint8, device="cuda")
        if c["op"] in ("fork", "compact"):
            m = s["meta"]
            h["pages"] = qb.KvPages(c["page"], m["nfree"], m["free"], m["refs"], m["lens"], m["tables"])
            h["ws"] = torch.empty(qb.kv_pages_workspace_bytes(h["pages"]), dtype=torch.uint8, device="cuda")
    if c["op"] == "append":
        qb.kv4_append(h["cache"], s["k"], s["v"], s["slots"])
        qb.kv4_read(h["cache"], s["slots"], s["k_back"], s["v_back"])
        return {"k": s["k_back"], "v": s["v_back"]}
    if c["op"] == "attn":
        qb.kv4_attn(h["cache"], s["q"], h["seqs"], c["d"] ** -0.5, s["out"], lse=s["lse"], window=c["window"], workspace=h["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    pages = h["pages"]
    s["state"].copy_(s["saved"])
    qb.kv_pages_free(pages, s["ended"])
    if c["op"] == "compact":
        qb.kv_pages_compact(pages, s["pool"], workspace=h["ws"])
        return {"state": s["state"], "pool": s["pool"]}
    qb.kv_pages_fork(pages, s["pool"], s["parents"], s["ended"], s["forked"], workspace=h["ws"])
    qb.kv_pages_extend(pages, s["all"], s["ones"], s["slots"], s["status"])
    return {"state": s["state"], "pool": s["pool"], "slots": s["slots"], "status": s["status"], "forked": s["forked"]}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """append: each group's step is its element of largest magnitude (the positive one where two are equal) over -8, rounded to f16; a code the nearest whole
    number, ties to even, of the element times the step's f32 reciprocal (a product rounded to f32), kept in -8..7; what is read is code times step.
    attn: softmax(q k' / sqrt(d)) v over the keys at or before each token's own place (and within the window), the elements taken from the cache one byte at a time."""
    c = case
    if c["op"] not in ("append", "attn"):
        return None
    s = prepare(case, seed)
    dp, page, nkv, d = _padded(c["d"]), c["page"], c["nkv"], c["d"]
    if c["op"] == "append":
        got = {}
        for name in "kv":
            x = s[name].double()
            x = torch.cat((x, x.new_zeros(*x.shape[:-1], -d % 32)), -1).reshape(*x.shape[:-1], -1, 32)
            big = x.abs().amax(-1, keepdim=True)
            plus = (x == big).any(-1, keepdim=True)
            step = (torch.where(plus, big, -big) / -8).half().double()
            inv = (1 / step).float().double()
            code = torch.round((x * inv).float().double()).clamp(-8, 7)
            code = torch.where(step == 0, 0.0, code)
            got[name] = (code * step).flatten(-2)[..., :d]
        return got
    lens, news = _lengths(c)
    if max(lens) * nkv * dp * 32 > 100e9 or max(n * t for n, t in zip(lens, news)) * c["nh"] * 24 > 100e9:
        return None
    w, bb = min(dp // 32, 4), _block_bytes(page, d)
    i = torch.arange(d, device="cuda")
    plane, g, e = i // 128, i // 32 % 4, i % 32
    code_bytes, step_bytes = page * dp // 2, page * dp // 16
    out, lse, at = [], [], 0
    for b, (n, t) in enumerate(zip(lens, news)):
        q = s["q"][at:at + t].double().reshape(t, nkv, -1, d)
        at += t
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
                flat = s["pool"].reshape(-1)
                code = (flat[o + byte].int() >> (4 * odd)) & 15
                lo = o + area + code_bytes + r * (dp // 16) + i // 32 * 2
                bits = flat[lo].int() | flat[lo + 1].int() << 8
                step = bits.to(torch.int16).view(torch.float16).double()
                heads.append((code - 8).double() * step)
            sides.append(torch.stack(heads))
        k, v = sides
        z = torch.einsum("thgd,hnd->thgn", q, k) / math.sqrt(d)
        pos = (n - t + torch.arange(t, device="cuda"))[:, None]
        seen = key[None] <= pos
        if c["window"]:
            seen &= key[None] > pos - c["window"]
        z = torch.where(seen[:, None, None, :], z, -math.inf)
        total = torch.logsumexp(z, -1) if n else z.new_full((t, nkv, c["nh"] // nkv), -math.inf)
        p = torch.where(torch.isfinite(total)[..., None], torch.exp(z - total[..., None]), 0.0)
        out.append(torch.einsum("thgn,hnd->thgd", p, v).reshape(t, -1, d))
        lse.append(total.reshape(t, -1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
