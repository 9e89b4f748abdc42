"""Inputs and 64-bit references of the operators on ragged batches of new tokens (no code of the library)."""
import numpy as np

D = 128
NAN = np.float16(np.nan)


def starts(lens):
    return np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)


def paged(lens, hkv, page, rng, spare=3, width=None):
    """Pools whose every slot that no sequence uses is NaN, and the page table (-1 behind the pages in use)."""
    need = [-(-c // page) for _, c in lens]
    pages = sum(need) + spare
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(max(need), 1) if width is None else width), -1, dtype=np.int32)
    k = np.full((pages, hkv, page, D), NAN, dtype=np.float16)
    v = k.copy()
    at = 0
    for b, (_, c) in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        for j in range(need[b]):
            fill = min(page, c - j * page)
            for pool in (k, v):
                pool[table[b, j], :, :fill] = rng.standard_normal((hkv, fill, D)).astype(np.float16)
    return k, v, table


def rows_of(pool, table_row, ctx, page):
    """[ctx][Hkv][D] in token order."""
    t = np.arange(ctx)
    return pool[table_row[t // page], :, t % page]


def attention(q, k, v, table, lens, page, window=0, scale=None):
    """(out, bound) in 64 bits: the attention of every row, and how far an fp16 result with P rounded to fp16 may be
    from it.

    The kernel's sums are in fp32 and P = exp(s - m) is rounded to fp16, m at most 8 (in powers of two) below the row's
    maximum and its own P being 1, so with A = sum p |v|:
      * rounding P is off by half a step, 2^-11 A, and by 2^-25 sum |v| / l, l >= 1, where P is subnormal;
      * a score is a sum of 128 products: off by at most 128 * 2^-23 * sum |q k| * scale =: e, which moves P and the sum of
        P by e each: 2 e A;
      * sums of P V and of P over the positions and the parts of a split: each term passes fewer than 2^9 additions
        (tiles, parts) and one tile's 128, 2^-23 each at most: 2 * 640 * 2^-23 A = 2^-13 A rounded up;
      * the result is rounded once, 2^-11 |out| (and 2^-25 where it is subnormal)."""
    T, hq, _ = q.shape
    g = hq // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, bound = np.zeros((T, hq, D)), np.zeros((T, hq, D))
    s0 = starts(lens)
    for b, (n, ctx) in enumerate(lens):
        if n == 0 or ctx <= 0:
            continue
        kk, vv = (rows_of(p, table[b], ctx, page).astype(np.float64) for p in (k, v))
        for h in range(hq):
            kh, vh = kk[:, h // g], vv[:, h // g]
            for i in range(n):
                pos = ctx - n + i
                if pos < 0:
                    continue
                lo = max(0, pos - window + 1) if window else 0
                x = q[s0[b] + i, h].astype(np.float64)
                s = kh[lo:pos + 1] @ x * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                a = p @ np.abs(vh[lo:pos + 1])
                e = 128 * 2.0 ** -23 * scale * (np.abs(kh[lo:pos + 1]) @ np.abs(x)).max()
                o = p @ vh[lo:pos + 1]
                out[s0[b] + i, h] = o
                bound[s0[b] + i, h] = (2.0 ** -11 * (a + np.abs(o)) + 2 * e * a + 2.0 ** -13 * a
                                      + 2.0 ** -25 * (np.abs(vh[lo:pos + 1]).sum(0) + 1))
    return out, bound


def frequencies(rd, theta, scaling="none", factor=1.0, original=0):
    """(angles a position, factor on cos and sin) in 64 bits."""
    f = theta ** (-2.0 * np.arange(rd // 2) / rd)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        turns = [rd * np.log(original / (r * 2 * np.pi)) / (2 * np.log(theta)) for r in (32, 1)]
        lo, hi = max(np.floor(turns[0]), 0), min(np.ceil(turns[1]), rd - 1)
        r = np.clip((np.arange(rd // 2) - lo) / (hi - lo), 0, 1)
        return f / factor * r + f * (1 - r), 0.1 * np.log(factor) + 1
    return f, 1.0


def rotate(x, pos, f, m, interleaved):
    """x [..., 128] with its first 2 len(f) values rotated at position pos, in 64 bits."""
    x = x.astype(np.float64)
    rd = 2 * len(f)
    y = x.copy()
    c, s = m * np.cos(pos * f), m * np.sin(pos * f)
    a, b = (slice(0, rd, 2), slice(1, rd, 2)) if interleaved else (slice(0, rd // 2), slice(rd // 2, rd))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


class PagesModel:
    """The pages of a cache in plain Python: the same requests give the same pages."""

    def __init__(self, table, ctx, refs, pools, page):
        self.table, self.ctx, self.refs = table.copy(), ctx.copy(), refs.copy()
        self.pools, self.page = pools.copy(), page  # [n_pools][pages][Hkv][page][D]

    def held(self, s):
        return min(-(-max(int(self.ctx[s]), 0) // self.page), self.table.shape[1])

    def free_pages(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def reserve(self, seqs, add):
        status, seen, free, at = [], set(), self.free_pages(), 0
        for s, a in zip(seqs, add):
            if s < 0 or s >= len(self.ctx) or s in seen or a < 0 or self.ctx[s] + a > self.table.shape[1] * self.page:
                status.append(2)
                seen.add(s)
                continue
            seen.add(s)
            old, new = self.held(s), -(-int(self.ctx[s] + a) // self.page)
            first, at = at, at + new - old
            if new > old and at > len(free):
                status.append(1)
                continue
            for j in range(new - old):
                self.table[s, old + j] = free[first + j]
                self.refs[free[first + j]] = 1
            self.ctx[s] += a
            status.append(0)
        return status

    def release(self, s):
        for p in self.table[s, :self.held(s)]:
            self.refs[p] -= 1
        self.table[s], self.ctx[s] = -1, 0

    def fork(self, src, dst):
        n, seen, status = len(self.ctx), {}, []
        for i, d in enumerate(dst):
            seen.setdefault(int(d), i)
        good = [0 <= s < n and 0 <= d < n and seen[int(d)] == i and int(s) not in seen
                for i, (s, d) in enumerate(zip(src, dst))]
        pairs = [(int(s), int(d)) if ok else None for s, d, ok in zip(src, dst, good)]
        for p in pairs:
            if p:
                self.release(p[1])
        for p in pairs:
            if p:
                for j in range(self.ctx[p[0]] // self.page):
                    self.refs[self.table[p[0], j]] += 1
        free, at = self.free_pages(), 0
        for p in pairs:
            if p is None:
                status.append(2)
                continue
            s, d = p
            full, fill = divmod(int(self.ctx[s]), self.page)
            if fill and at >= len(free):
                status.append(1)
                for j in range(full):
                    self.refs[self.table[s, j]] -= 1
                continue
            self.table[d, :full] = self.table[s, :full]
            if fill:
                new = free[at]
                at += 1
                self.refs[new] = 1
                self.table[d, full] = new
                self.pools[:, new, :, :fill] = self.pools[:, self.table[s, full], :, :fill]
            self.ctx[d] = self.ctx[s]
            status.append(0)
        return status

    def compact(self):
        live = [p for p in range(len(self.refs)) if self.refs[p] > 0]
        n = len(live)
        gaps = [p for p in range(n) if self.refs[p] == 0]
        move = dict(zip([p for p in live if p >= n], gaps))
        for a, b in move.items():
            self.pools[:, b] = self.pools[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for s in range(len(self.ctx)):
            for j in range(self.held(s)):
                self.table[s, j] = move.get(int(self.table[s, j]), self.table[s, j])
        return n
