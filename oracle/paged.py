"""The paged KV cache's operators restated plainly on the host: numpy in 64 bits for what is computed, the fp32 steps of
the definition where results are fixed bit for bit, Python lists for the page tables. Shares no code with the library."""
import numpy as np


def bf16(x):
    """fp32 array rounded to bfloat16 (nearest even), as fp32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r).reshape(np.shape(x))


def values(codes, scales):
    """What 8-bit cache elements stand for: fp16(scale * code), in fp64. codes [..., D], scales [..., D / 32]."""
    wide = np.repeat(scales.astype(np.float64), 32, -1)
    with np.errstate(over="ignore"):
        return (codes.astype(np.float64) * wide).astype(np.float16).astype(np.float64)


def rotate32(x, rope_rows):
    """The rotation in the definition's fp32 steps. x [n, H, D] fp32, rope_rows [n, D] fp32."""
    h = x.shape[-1] // 2
    c, s = rope_rows[:, None, :h], rope_rows[:, None, h:]
    a, b = x[..., :h], x[..., h:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1).astype(np.float32)


def rotate64(x, rope_rows):
    """The rotation's formula in fp64."""
    h = x.shape[-1] // 2
    ang = rope_rows.astype(np.float64)[:, None, :]
    z = (x[..., :h] + 1j * x[..., h:].astype(np.float64)) * (ang[..., :h] + 1j * ang[..., h:])
    return np.concatenate([z.real, z.imag], -1)


def quantize32(x):
    """8-bit rule on fp32 [..., D], the definition's fp32 steps: (codes int8, scales fp16)."""
    g = x.astype(np.float32).reshape(x.shape[:-1] + (-1, 32))
    m = np.abs(g).max(-1)
    d16 = np.minimum(m / np.float32(127), np.float32(65504)).astype(np.float16)
    d = d16.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.clip(np.rint(g / d), -127, 127)
    return np.where(d > 0, q, 0).astype(np.int8).reshape(x.shape), d16


def attend(q, k, v, scale, window=0, rope_row=None):
    """One row. q [Hq, D], k and v [L, H, D], fp64. Returns out [Hq, D], lse [Hq]."""
    Hq, D = q.shape
    L, H = k.shape[0], v.shape[1]
    if L == 0:
        return np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if rope_row is not None:
        q = rotate64(q[None], rope_row[None])[0]
    lo = max(0, L - window) if window else 0
    k, v = k[lo:], v[lo:]
    out, lse = np.empty((Hq, D)), np.empty(Hq)
    for h in range(Hq):
        kv = h // (Hq // H)
        x = (k[:, kv] @ q[h]) * scale
        m = x.max()
        e = np.exp(x - m)
        out[h] = (e[:, None] * v[:, kv]).sum(0) / e.sum()
        lse[h] = m + np.log(e.sum())
    return out, lse


class Pages:
    """Page tables by the definition of the page operators; `pool` is any numpy array [pages, tokens, ...] moved along."""

    def __init__(self, seqs, max_pages, pages, tokens, pool=None):
        self.T, self.P, self.MP = tokens, pages, max_pages
        self.tables = [[-1] * max_pages for _ in range(seqs)]
        self.lens, self.refs = [0] * seqs, [0] * pages
        self.pool = pool
        self.refused = self.bad = False

    def free_pages(self):
        return [p for p in range(self.P) if self.refs[p] == 0]

    def reserve(self, seqs, add):
        free, used = self.free_pages(), 0
        for s, n in zip(seqs, add):
            if s < 0:
                continue
            old, new = -(-self.lens[s] // self.T), -(-(self.lens[s] + n) // self.T)
            if new > self.MP:
                self.refused = True
                continue
            take = free[used:used + new - old]
            used += new - old
            if len(take) < new - old:
                self.refused = True
                continue
            self.tables[s][old:new] = take
            for p in take:
                self.refs[p] = 1
            self.lens[s] += n

    def fork(self, src, dst):
        free, used = self.free_pages(), 0
        for s, d in zip(src, dst):
            full, rows = divmod(self.lens[s], self.T)
            fresh = None
            if rows:
                fresh = free[used] if used < len(free) else None
                used += 1
            if self.lens[d] != 0 or (rows and fresh is None):
                self.refused = True
                continue
            for c in range(full):
                self.tables[d][c] = self.tables[s][c]
                self.refs[self.tables[s][c]] += 1
            if rows:
                self.tables[d][full] = fresh
                self.refs[fresh] = 1
                if self.pool is not None:
                    self.pool[fresh][:rows] = self.pool[self.tables[s][full]][:rows]
            self.lens[d] = self.lens[s]

    def free(self, seqs):
        for s in seqs:
            if s < 0:
                continue
            for c, p in enumerate(self.tables[s]):
                if p >= 0:
                    self.refs[p] -= 1
                    self.tables[s][c] = -1
            self.lens[s] = 0

    def compact(self):
        live = [p for p in range(self.P) if self.refs[p] > 0]
        n = len(live)
        movers = [p for p in live if p >= n]
        holes = [p for p in range(n) if self.refs[p] <= 0]
        new = dict(zip(movers, holes))
        for a, b in new.items():
            if self.pool is not None:
                self.pool[b] = self.pool[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.tables = [[new.get(p, p) for p in row] for row in self.tables]
        return len(movers)
