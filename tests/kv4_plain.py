"""The 4-bit KV cache in plain numpy / 64-bit arithmetic, for the tests: the format, a pool written byte
by byte, attention row by row, and eviction.  Shares no code with the library."""
import numpy as np

BLOCK = 32


def quantize(x):
    """x fp32 [..., d] -> codes int [..., d], scale and lo fp16 [..., d / 64]."""
    g = np.clip(np.asarray(x, np.float32), -65504.0, 65504.0).reshape(x.shape[:-1] + (-1, 64))
    with np.errstate(all="ignore"):
        lo32, hi32 = g.min(-1), g.max(-1)  # NaN if there is one
        lo = lo32.astype(np.float16)
        scale = ((hi32 - lo32) / np.float32(15)).astype(np.float16)
        s32, l32 = scale.astype(np.float32)[..., None], lo.astype(np.float32)[..., None]
        q = np.where(s32 > 0, (g - l32) / np.where(s32 > 0, s32, np.float32(1)), np.float32(0))
    code = np.clip(np.rint(q), 0, 15).astype(np.int64)
    return code.reshape(x.shape), scale, lo


def values(code, scale, lo):
    """What the rows stand for, in 64 bits."""
    g = code.reshape(code.shape[:-1] + (-1, 64)).astype(np.float64)
    return (lo.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * g).reshape(code.shape)


class PlainPool:
    """A pool of pages as bytes; every byte is garbage (0xff: NaN scales, negative positions) until written."""

    def __init__(self, n_layers, n_kv, d, num_pages, page, track):
        self.L, self.nkv, self.d, self.page, self.track = n_layers, n_kv, d, page, track
        self.code, self.pair = BLOCK * d // 2, BLOCK * (d // 64) * 4
        self.block = 2 * (self.code + self.pair) + (256 if track else 0)
        self.bytes = np.full((num_pages, n_layers, n_kv, page // BLOCK, self.block), 0xFF, np.uint8)

    def _at(self, table, row):
        return int(table[row // self.page]), row % self.page // BLOCK, row % BLOCK

    def put(self, layer, table, row, h, k, v, pos=None, weight=0.0):
        """Row `row` of the sequence with page table `table`, KV head h, from fp32 k and v [d]."""
        page, b, r = self._at(table, row)
        blk = self.bytes[page, layer, h, b]
        for sel, x in ((0, k), (1, v)):
            base, n = sel * (self.code + self.pair), self.d // 64
            code, scale, lo = quantize(x)
            blk[base + r * self.d // 2: base + (r + 1) * self.d // 2] = (code[0::2] | code[1::2] << 4).astype(np.uint8)
            at = base + self.code + r * n * 4
            blk[at:at + 4 * n] = np.stack([scale, lo], -1).reshape(-1).view(np.uint8)
        if self.track:
            at = 2 * (self.code + self.pair)
            blk[at + 4 * r:at + 4 * r + 4] = np.array([pos], np.int32).view(np.uint8)
            blk[at + 128 + 4 * r:at + 132 + 4 * r] = np.array([weight], np.float32).view(np.uint8)

    def get(self, layer, table, row, h):
        """(k, v) in 64 bits."""
        page, b, r = self._at(table, row)
        blk, out = self.bytes[page, layer, h, b], []
        for sel in (0, 1):
            base, n = sel * (self.code + self.pair), self.d // 64
            byte = blk[base + r * self.d // 2: base + (r + 1) * self.d // 2].astype(np.int64)
            code = np.stack([byte & 15, byte >> 4], -1).reshape(-1)
            p = blk[base + self.code + r * n * 4: base + self.code + (r + 1) * n * 4].copy().view(np.float16).reshape(n, 2)
            out.append(values(code, p[:, 0], p[:, 1]))
        return out

    def _word(self, layer, table, row, h, at, dtype):
        page, b, r = self._at(table, row)
        at += 2 * (self.code + self.pair) + 4 * r
        return self.bytes[page, layer, h, b, at:at + 4].copy().view(dtype)[0]

    def pos(self, layer, table, row, h):
        return int(self._word(layer, table, row, h, 0, np.int32)) if self.track else row

    def weight(self, layer, table, row, h):
        return float(self._word(layer, table, row, h, 128, np.float32))

    def row_bytes(self, layer, table, row, h):
        """Everything that belongs to a row, as one array of bytes."""
        page, b, r = self._at(table, row)
        blk, n, part = self.bytes[page, layer, h, b], self.d // 64 * 4, []
        for sel in (0, 1):
            base = sel * (self.code + self.pair)
            part += [blk[base + r * self.d // 2: base + (r + 1) * self.d // 2], blk[base + self.code + r * n: base + self.code + (r + 1) * n]]
        at = 2 * (self.code + self.pair)
        return np.concatenate(part + [blk[at + 4 * r:at + 4 * r + 4], blk[at + 128 + 4 * r:at + 132 + 4 * r]])


def attention(pool, layer, q, offsets, rows, tables, positions, n_heads, scale, cap=0.0, slopes=None, window=0):
    """(out [n, heads, d], {(sequence, row, head): weight}) in 64 bits; rows that see nothing are zero."""
    q = np.asarray(q, np.float64)
    out, weights, g = np.zeros_like(q), {}, n_heads // pool.nkv
    for s, r in enumerate(rows):
        c = offsets[s + 1] - offsets[s]
        if c == 0:
            continue
        p0 = positions[s] if positions is not None else r - c
        for h in range(pool.nkv):
            kv = [pool.get(layer, tables[s], i, h) for i in range(r)]
            k = np.array([x[0] for x in kv]).reshape(r, pool.d)
            v = np.array([x[1] for x in kv]).reshape(r, pool.d)
            kpos = np.array([pool.pos(layer, tables[s], i, h) for i in range(r)], np.int64)
            total = np.zeros(r)
            for i in range(c):
                see = np.arange(r) <= r - c + i
                if window:
                    see &= (p0 + i) - kpos < window
                if not see.any():
                    continue
                for j in range(h * g, (h + 1) * g):
                    x = (k[see] @ q[offsets[s] + i, j]) * scale
                    if cap:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        x = x + float(slopes[j]) * (kpos[see] - (p0 + i))
                    e = np.exp(x - x.max())
                    p = e / e.sum()
                    out[offsets[s] + i, j] = p @ v[see]
                    total[see] += p
            for i in range(r):
                weights[s, i, h] = total[i]
    return out, weights


def evict_map(weights, pos, keep, young):
    """Source row of each row that is left."""
    r = len(weights)
    if r <= keep:
        return list(range(r))
    order = sorted(range(r), key=lambda i: (pos[i] < young, 0.0 if pos[i] >= young else -(0.0 if np.isnan(weights[i]) else weights[i]), i))
    kept = set(order[:keep])
    above = iter(sorted(i for i in kept if i >= keep))
    return [i if i in kept else next(above) for i in range(keep)]
