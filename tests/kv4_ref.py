"""The paged 4-bit cache and its operators in plain numpy: bytes as the header's
layout has them, quantization in f32 as it is defined, attention in 64 bits,
pages with lists."""
import numpy as np


def padded(d):
    return 64 if d <= 64 else 128 if d <= 128 else 256


def block_bytes(page, d):
    dp = padded(d)
    return 2 * page * (dp // 2 + dp // 16)


def key_nibble(page, dp, r, i):
    w, G, e = min(dp // 32, 4), i // 32, i % 32
    return ((((G // 4) * page + r) * 4 + e // 8) * w + G % 4) * 8 + e % 8


def value_nibble(page, dp, r, i):
    w, G, e = min(dp // 32, 4), i // 32, i % 32
    chunk = (e // 4) ^ (4 * ((r >> 1) & 1))
    return ((((G // 4) * page + r) * 8 + chunk) * w + G % 4) * 4 + e % 4


def quantize(x):
    """x f32 [..., dp] -> codes uint8 0..15, steps f16 [..., dp/32]."""
    g = x.reshape(*x.shape[:-1], -1, 32).astype(np.float32)
    finite = np.where(np.isnan(g), np.float32(0), g)
    hi = np.maximum(finite.max(-1), 0)
    lo = np.minimum(finite.min(-1), 0)
    with np.errstate(all="ignore"):
        step = (np.where(hi >= -lo, hi, lo).astype(np.float32) * np.float32(-0.125)).astype(np.float16)
        s = step.astype(np.float32)
        inv = np.where(s == 0, np.float32(0), np.float32(1) / np.where(s == 0, np.float32(1), s)).astype(np.float32)
        prod = (g * inv[..., None]).astype(np.float32)
        code = np.where(np.isnan(prod), 0, np.clip(np.rint(prod), -8, 7)) + 8
    return code.astype(np.uint8).reshape(x.shape), step


def dequantize(codes, step):
    with np.errstate(invalid="ignore"):
        return ((codes.reshape(*codes.shape[:-1], -1, 32).astype(np.float64) - 8) *
                step.astype(np.float64)[..., None]).reshape(codes.shape)


def _set_nibbles(area, nibs, codes):
    for n, c in zip(nibs, codes):
        b = area[n // 2]
        area[n // 2] = (b & 0xF0) | c if n % 2 == 0 else (b & 0x0F) | (c << 4)


def write_row(pool, page, nkv, d, slot, k, v):
    """k, v f32 [nkv, d] into pool uint8 [npages, nkv * block_bytes]."""
    dp = padded(d)
    pg, r = divmod(int(slot), page)
    bb, cb, sb = block_bytes(page, d), page * dp // 2, page * dp // 16
    i = np.arange(dp)
    for h in range(nkv):
        block = pool[pg, h * bb:(h + 1) * bb]
        for x, at, nib in ((k, 0, key_nibble(page, dp, r, i)), (v, cb + sb, value_nibble(page, dp, r, i))):
            row = np.zeros(dp, np.float32)
            row[:d] = x[h]
            codes, step = quantize(row)
            _set_nibbles(block[at:at + cb], nib, codes)
            block[at + cb + r * (dp // 16):at + cb + (r + 1) * (dp // 16)] = step.view(np.uint8)


def read_row(pool, page, nkv, d, slot):
    """The values at a slot: k, v f64 [nkv, d]."""
    dp = padded(d)
    pg, r = divmod(int(slot), page)
    bb, cb, sb = block_bytes(page, d), page * dp // 2, page * dp // 16
    i = np.arange(dp)
    out = np.zeros((2, nkv, d))
    for h in range(nkv):
        block = pool[pg, h * bb:(h + 1) * bb]
        for side, (at, nib) in enumerate(((0, key_nibble(page, dp, r, i)), (cb + sb, value_nibble(page, dp, r, i)))):
            area = block[at:at + cb]
            codes = (area[nib // 2] >> (4 * (nib % 2))) & 15
            step = block[at + cb + r * (dp // 16):at + cb + (r + 1) * (dp // 16)].copy().view(np.float16)
            out[side, h] = dequantize(codes, step)[:d]
    return out[0], out[1]


def attention(q, rows_k, rows_v, n, T, scale, window):
    """q f64 [T, nh, d]; rows_k, rows_v f64 [n, nkv, d] -> out, lse, and for tolerances: the largest sum of magnitudes
    in a score [T, nh] and the softmax-weighted magnitudes of the values [T, nh, d]."""
    nh, d = q.shape[1:]
    grp = nh // rows_k.shape[1] if n else 1
    out, mag = np.zeros((T, nh, d)), np.zeros((T, nh, d))
    lse, zabs = np.full((T, nh), -np.inf), np.zeros((T, nh))
    for j in range(T):
        pos = n - T + j
        first = max(0, pos - window + 1) if window else 0
        if pos < first:
            continue
        for h in range(nh):
            k, v = rows_k[first:pos + 1, h // grp], rows_v[first:pos + 1, h // grp]
            with np.errstate(invalid="ignore"):
                z = scale * (k @ q[j, h])
                zabs[j, h] = np.max(abs(scale) * (np.abs(k) @ np.abs(q[j, h])))
                m = z.max()
                e = np.exp(z - m)
                lse[j, h] = m + np.log(e.sum())
                p = e / e.sum()
                out[j, h] = p @ v
                mag[j, h] = p @ np.abs(v)
    return out, lse, zabs, mag


class Pages:
    """The pages' state with lists."""

    def __init__(self, page, npages, nrows, maxp, layers=1, pool=None):
        self.page, self.npages, self.nrows, self.maxp = page, npages, nrows, maxp
        self.stack = list(range(npages - 1, -1, -1))
        self.refs = [0] * npages
        self.rows = [[] for _ in range(nrows)]
        self.lens = [0] * nrows
        self.pool = pool  # [layers, npages, bytes]

    def extend(self, rows, counts):
        status, slots, left = [], [], len(self.stack)
        for r, c in zip(rows, counts):
            if c < 0 or not 0 <= r < self.nrows:
                status.append(-1)
                slots += [-1] * max(c, 0)
                continue
            if self.lens[r] + c > self.maxp * self.page:
                status.append(-8)
                slots += [-1] * c
                continue
            need = -(-(self.lens[r] + c) // self.page) - len(self.rows[r])
            left -= need
            if need and left < 0:
                status.append(-8)
                slots += [-1] * c
                continue
            for _ in range(need):
                pg = self.stack.pop()
                self.refs[pg] = 1
                self.rows[r].append(pg)
            for t in range(self.lens[r], self.lens[r] + c):
                slots.append(self.rows[r][t // self.page] * self.page + t % self.page)
            self.lens[r] += c
            status.append(0)
        return slots, status

    def fork(self, parents, children):
        status = []
        for p, c in zip(parents, children):
            if not (0 <= p < self.nrows and 0 <= c < self.nrows) or self.lens[c]:
                status.append(-1)
                continue
            tail = self.lens[p] % self.page
            if tail and not self.stack:
                status.append(-8)
                continue
            row = list(self.rows[p])
            for pg in row[:len(row) - bool(tail)]:
                self.refs[pg] += 1
            if tail:
                pg = self.stack.pop()
                self.refs[pg] = 1
                if self.pool is not None:
                    self.pool[:, pg] = self.pool[:, row[-1]]
                row[-1] = pg
            self.rows[c], self.lens[c] = row, self.lens[p]
            status.append(0)
        return status

    def free(self, rows):
        back = []
        for r in rows:
            if not 0 <= r < self.nrows:
                continue
            for pg in self.rows[r]:
                self.refs[pg] -= 1
                if self.refs[pg] == 0:
                    back.append(pg)
            self.rows[r], self.lens[r] = [], 0
        self.stack += sorted(back)

    def compact(self):
        held = [i for i in range(self.npages) if self.refs[i]]
        used = len(held)
        moves = dict(zip([i for i in held if i >= used], [i for i in range(used) if not self.refs[i]]))
        for a, b in moves.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
            if self.pool is not None:
                self.pool[:, b] = self.pool[:, a]
        self.rows = [[moves.get(x, x) for x in r] for r in self.rows]
        self.stack = list(range(self.npages - 1, used - 1, -1))
