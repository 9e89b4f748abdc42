"""Attention of new tokens where its numbers are hard: weights far below the row's largest, scores of any finite size, rows
summed again in parts of a cut unit, the longest row (needs a B200)."""
import numpy as np
import pytest

import chunk_cases as cc
from helpers import dev

pytestmark = pytest.mark.gpu


def put(pool, table, b, t, value):
    """Position t of sequence b, all kv heads."""
    page = pool.shape[2]
    pool[table[b, t // page], :, t % page] = value


def call(i4, cuda, q, k, v, table, lens, **kw):
    import torch
    got = i4.paged_gqa_chunk(dev(q, cuda), dev(k, cuda), dev(v, cuda), dev(table, cuda), dev(cc.starts(lens), cuda),
                             dev(np.array([c for _, c in lens], dtype=np.int32), cuda), **kw)
    torch.cuda.synchronize()
    assert i4.device_error() == 0
    return got.cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ weights far below the largest

@pytest.mark.parametrize("n,ctx,hkv", [(1, 32768, 1), (5, 32768, 1), (300, 32768, 1), (1, 1 << 17, 1), (1024, 6144, 16)])
@pytest.mark.parametrize("key", [24.5625, 24.0, 27.0])
@pytest.mark.parametrize("place", [0, 0.5, 1])
def test_a_dominant_position_leaves_the_others_their_share(i4lib, cuda, n, ctx, hkv, key, place):
    """One position whose weight is about 2^25 (2^24.5, 2^27.5) times that of each other one, and whose V is 0: the output is
    what the others have together. q = 8 and K = `key` in the first dim, everything else 0, so every score is exact, and a row
    that sees N other positions has w v N / (1 + N w) in all, w = 2^(-8 key / sqrt(128) log2(e)). The last shape's units are whole
    (one maximum for the row), the others' are cut: parts without the position have a maximum of their own.

    P is held in fp16 as 2^7 times the weight relative to the row's m, which is at most the maximum: off by half a step,
    2^-11 of it, or by 2^-25 / 2^7 = 2^-32 of the largest weight where it is subnormal. One more 2^-11 rounds the result (2^-25
    where that is subnormal), 2^-13 its sums, and exp's argument is off by 2^-19 (that of a number below 64 in fp32, times
    log 2), as its approximation is by 2^-22."""
    lens, page = [(n, ctx)], 64
    pages = ctx // page
    table = np.random.default_rng(ctx).permutation(pages).astype(np.int32)[None]
    k, v = (np.zeros((pages, hkv, page, cc.D), dtype=np.float16) for _ in range(2))
    v[:] = np.arange(1, cc.D + 1, dtype=np.float16) / 64
    sink = int(place * (ctx - n))  # seen by every row
    value = np.zeros(cc.D, dtype=np.float16)
    value[0] = key
    put(k, table, 0, sink, value)
    put(v, table, 0, sink, np.zeros(cc.D, dtype=np.float16))
    q = np.zeros((n, 4 * hkv, cc.D), dtype=np.float16)
    q[:, :, 0] = 8
    got = call(i4lib, cuda, q, k, v, table, lens)
    w = np.exp(-8 * key / np.sqrt(128))
    others = (ctx - n + np.arange(n)).astype(np.float64)[:, None, None]  # row i sees ctx - n + i beside the sink
    v0 = np.arange(1, cc.D + 1) / 64
    want = others * w * v0 / (1 + others * w)
    bound = want * (2.0 ** -10 + 2.0 ** -13 + 2.0 ** -18) + others * 2.0 ** -32 * v0 + 2.0 ** -25
    assert np.all(bound < want / 4)  # a result without the others' share would show
    assert np.all(np.abs(got - want) <= bound), (got[0, 0, :4], want[0, 0, :4])


# ------------------------------------------------------------------ scores of any finite size

def needle_case(n, ctx, size, seed, sign=1):
    """Signs times `size` in q (one pattern for all rows), K = a fraction of the pattern times `size`: position `top` has the
    greatest score by more than 2^-9 of it, so its weight is 1 and every other one 0 wherever the scores differ by more than
    2^7."""
    rng = np.random.default_rng(seed)
    page = 16
    lens = [(n, ctx)]
    k, v, table = cc.paged(lens, 1, page, rng)
    pattern = rng.choice([-1.0, 1.0], size=cc.D)
    q = np.broadcast_to(np.float16(size * pattern), (n, 4, cc.D)).copy()
    part = rng.integers(128, 384, size=ctx) / 512.0  # of 512ths: products of powers of two and small integers, exact
    top = ctx - n - 1 if seed % 2 else int(rng.integers(0, ctx - n))
    part[top] = 0.8125 if sign > 0 else 0.125
    for t in range(ctx):
        put(k, table, 0, t, np.float16(sign * part[t] * size * pattern))
    return lens, q, k, v, table, top


@pytest.mark.parametrize("n,ctx", [(1, 5000), (3, 700), (300, 1300), (1, 60)])
@pytest.mark.parametrize("size", [64.0, 512.0, 4096.0, 32768.0])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(i4lib, cuda, n, ctx, size, sign):
    """Scores up to 2^37 and their negatives: the row's largest takes everything. Its V is multiplied by a P of 2^7 to 2^15
    rounded to fp16 (2^-11), divided by their sum and rounded (2^-11); the sums are fp32 (2^-13 covers them)."""
    lens, q, k, v, table, top = needle_case(n, ctx, size, seed=n + ctx, sign=sign)
    got = call(i4lib, cuda, q, k, v, table, lens)
    want = cc.rows_of(v, table[0], ctx, 16)[top, 0].astype(np.float64)
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -10 + 2.0 ** -13) + 2.0 ** -25)


@pytest.mark.parametrize("scale", [1e6, 1e15, 1e20])
@pytest.mark.parametrize("n,ctx", [(1, 3000), (40, 300), (200, 400)])
def test_large_scale(i4lib, cuda, n, ctx, scale):
    """Ordinary q and K under a scale that makes every score huge: each row gives the V of its largest score, wherever the two
    largest differ by more than fp32 sums of 128 products may be off (128 * 2^-23 sum |q k| each)."""
    lens, page = [(n, ctx)], 32
    rng = np.random.default_rng(ctx)
    k, v, table = cc.paged(lens, 1, page, rng)
    q = rng.standard_normal((n, 4, cc.D)).astype(np.float16)
    got = call(i4lib, cuda, q, k, v, table, lens, scale=scale)
    assert np.all(np.isfinite(got))
    kk, vv = (cc.rows_of(p, table[0], ctx, page)[:, 0].astype(np.float64) for p in (k, v))
    seen = 0
    for i in range(n):
        s = kk[:ctx - n + i + 1] @ q[i].astype(np.float64).T
        for h in range(4):
            order = np.argsort(s[:, h])
            off = 2 * 128 * 2.0 ** -23 * (np.abs(kk[order[-2:]]) @ np.abs(q[i, h].astype(np.float64))).max()
            if s[order[-1], h] - s[order[-2], h] <= off + 130 / scale:
                continue
            seen += 1
            want = vv[order[-1]]
            assert np.all(np.abs(got[i, h] - want) <= np.abs(want) * (2.0 ** -10 + 2.0 ** -13) + 2.0 ** -25), (i, h)
    assert seen > 3 * n  # nearly every row has a clear maximum


@pytest.mark.parametrize("size", [64.0, 4096.0, 32768.0])
def test_equal_large_scores_share(i4lib, cuda, size):
    """Two positions far apart with the same, greatest score: the mean of their V, whichever part of a split each is in."""
    lens, q, k, v, table, top = needle_case(2, 9000, size, seed=8)
    other = 9000 - 3 - top if abs(9000 - 3 - 2 * top) > 2000 else (top + 4000) % 8990
    put(k, table, 0, other, cc.rows_of(k, table[0], 9000, 16)[top])
    vv = cc.rows_of(v, table[0], 9000, 16)[:, 0].astype(np.float64)
    got = call(i4lib, cuda, q, k, v, table, lens)
    want, a = (vv[top] + vv[other]) / 2, (np.abs(vv[top]) + np.abs(vv[other])) / 2
    assert np.all(np.abs(got - want) <= 2.0 ** -11 * (a + np.abs(want)) + 2.0 ** -13 * a + 2.0 ** -25)


def test_a_maximum_that_creeps_at_large_scores(i4lib, cuda):
    """Scores near 2^30 that rise by a step of their fp32 sum (16 to 128) from position to position: P stays finite though the
    maximum is followed late."""
    ctx, page = 2000, 16
    lens = [(1, ctx)]
    rng = np.random.default_rng(3)
    k, v, table = cc.paged(lens, 1, page, rng)
    q = np.zeros((1, 4, cc.D), dtype=np.float16)
    q[0, :, 0], q[0, :, 1] = 32768, 1
    for h in range(4):
        q[0, h, 1] = 2.0 ** (3 + h)
    for t in range(ctx):
        value = np.zeros(cc.D, dtype=np.float16)
        value[0], value[1] = 32768, t / 8 if t < 1900 else 0
        put(k, table, 0, t, value)
    got = call(i4lib, cuda, q, k, v, table, lens, scale=1.0)
    assert np.all(np.isfinite(got))
    kk, vv = (cc.rows_of(p, table[0], ctx, page)[:, 0].astype(np.float64) for p in (k, v))
    # the sums are rounded to steps of 2^(30-23) = 128: the weights are those of some scores within 128 of the exact ones, so
    # the output lies within the V of the positions that near the largest
    s = kk @ q[0].astype(np.float64).T
    for h in range(4):
        near = vv[s[:, h] >= s[:, h].max() - 2 * 128 - 20]
        slack = np.abs(near).max(0) * 2.0 ** -9 + 2.0 ** -20
        assert np.all(got[0, h] >= near.min(0) - slack) and np.all(got[0, h] <= near.max(0) + slack)


# ------------------------------------------------------------------ rows summed again in parts of a cut unit

@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 65504.0])
@pytest.mark.parametrize("lens,window", [
    ([(5, 20005)], 0), ([(40, 20040)], 0), ([(5, 20005)], 3000), ([(40, 9040), (5, 20005), (1, 700)], 2500),
    ([(60, 30000), (200, 12200)], 4000),
])
def test_what_a_row_does_not_see_in_a_cut_unit(i4lib, cuda, bad, lens, window):
    """Long contexts whose units are cut into parts: K and V of the last token, and of the tokens just before the last row's
    window, are NaN or infinite. Rows that see none of them are held to the bound, and no page lies in order."""
    rng = np.random.default_rng(len(lens) + window)
    k, v, table = cc.paged(lens, 1, 64, rng)
    q = rng.standard_normal((int(cc.starts(lens)[-1]), 7, cc.D)).astype(np.float16)
    clean, good, row = (k.copy(), v.copy()), [], 0
    for b, (n, ctx) in enumerate(lens):
        marked = {ctx - 1}
        if window:  # seen by the chunk's first row, not by the later ones; the first sees nothing else that is marked
            marked |= {ctx - n - window + 1} if ctx - n - window + 1 >= 0 else set()
        for t in marked:
            put(k, table, b, t, bad)
            put(v, table, b, t, bad)
        for i in range(n):
            pos = ctx - n + i
            if not any(t <= pos and (not window or t > pos - window) for t in marked):
                good.append(row + i)
        row += n
    got = call(i4lib, cuda, q, k, v, table, lens, window=window)
    want, bound = cc.attention(q, *clean, table, lens, 64, window)
    assert len(good) >= len(q) - 2 * len(lens)
    off = np.abs(got[good] - want[good]) - bound[good]
    assert np.all(np.isfinite(got[good])) and off.max() <= 0, off.max()


def test_rows_summed_again_beside_large_scores(i4lib, cuda):
    """Scores of 2^30 and a NaN in the last token's V: the other rows are summed again and still give their largest's V."""
    for n, ctx in ((3, 700), (6, 9000), (300, 1300)):
        lens, q, k, v, table, top = needle_case(n, ctx, 4096.0, seed=n + ctx)
        want = cc.rows_of(v, table[0], ctx, 16)[top, 0].astype(np.float64)
        put(v, table, 0, ctx - 1, np.nan)
        got = call(i4lib, cuda, q, k, v, table, lens)[:-1]
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -10 + 2.0 ** -13) + 2.0 ** -25)


# ------------------------------------------------------------------ the longest row

def longest_row(q, k, v, keep=None):
    """64-bit attention of q [Hq][128] over k, v, with what an fp16 result may be off: A and the weights from the reference
    itself. `keep` drops positions."""
    import torch
    s = q.double() @ k.double().T / np.sqrt(cc.D)
    if keep is not None:
        s = s.masked_fill(~keep, -float("inf"))
    p = torch.softmax(s, dim=1)
    out, a = p @ v.double(), p @ v.double().abs()
    e = 128 * 2.0 ** -23 / np.sqrt(cc.D) * (q.double().abs() @ k.double().abs().T).amax(dim=1, keepdim=True)
    tiny = p.amax(dim=1, keepdim=True) * 2.0 ** -32 * v.double().abs().sum(0)  # P below 2^-14, 2^7 times the weight
    # sums: 8192 tiles and parts, a tile's 128, 2^-23 each, of P V and of P
    bound = 2.0 ** -11 * (a + out.abs()) + 2 * e * a + 2 * (8192 + 128) * 2.0 ** -23 * a + tiny + 2.0 ** -25
    return out, bound


@pytest.mark.parametrize("n", [1, 2, 40])
def test_a_million_positions_by_value(i4lib, cuda, n):
    """The longest row of the page table, V with a mean, and one position in every 2^16 whose weight is some 3 % of all: a lost
    part or a zero would be far outside the bound, which the test shows first."""
    import torch
    ctx, page = 1 << 20, 128
    gen = torch.Generator(device=cuda).manual_seed(n)
    k, v = (torch.randn((ctx // page, 1, page, 128), generator=gen, device=cuda, dtype=torch.float16) for _ in range(2))
    v += 1
    perm = torch.randperm(ctx // page, generator=gen, device=cuda)
    q = torch.randn((n, 4, 128), generator=gen, device=cuda, dtype=torch.float16)
    q[:, :, 0] = 16
    for i in range(16):  # a score of 16 * 8.5 / sqrt(128) = 12 beside the other dims', and V far from the mean of all
        t = i * 65536 + 1000 + 3001 * i
        k[perm[t // page], 0, t % page, 0] = 8.5
        v[perm[t // page], 0, t % page] = 2.0 if i % 2 else 30.0
    table = perm.to(torch.int32)[None].contiguous()
    start, lens = torch.tensor([0, n], dtype=torch.int32, device=cuda), torch.tensor([ctx], dtype=torch.int32, device=cuda)
    got = i4lib.paged_gqa_chunk(q, k, v, table, start, lens, max_q=n).double()
    assert i4lib.device_error() == 0
    kk, vv = (t[perm][:, 0].reshape(-1, 128) for t in (k, v))
    for i in sorted({0, n // 2, n - 1}):
        sees = ctx - n + 1 + i
        want, bound = longest_row(q[i], kk[:sees], vv[:sees])
        assert bool((want.abs() > bound).all())  # zeros would show
        part = torch.arange(sees, device=cuda)
        for a in (0, 1 << 19, sees - 70000):  # and so would a stretch of 7000 positions with a planted one, left out for all heads
            a = a // 65536 * 65536 + 1000 + 3001 * (a // 65536) - 3500
            lost, _ = longest_row(q[i], kk[:sees], vv[:sees], keep=(part < a) | (part >= a + 7000))
            assert bool(((lost - want).abs() > 2 * bound).any())
        assert bool(((got[i] - want).abs() <= bound).all())


# ------------------------------------------------------------------ repeated calls, early launches off

@pytest.mark.parametrize("lens,hq,hkv,page,window", [
    ([(1, 514), (1, 77), (1, 1000), (1, 2049)], 28, 4, 16, 0),
    ([(512, 512)], 28, 4, 16, 0),
    ([(512, 9000)], 28, 4, 64, 0),
    ([(1, 4093), (301, 2348), (1, 17), (1, 8191), (777, 777), (64, 5000), (0, 100), (1, 1)], 32, 4, 32, 2000),
])
def test_every_call_gives_the_same_bits(i4lib, cuda, lens, hq, hkv, page, window):
    """Also without the early launches, and with other work on the GPU at the same time."""
    import torch
    rng = np.random.default_rng(1)
    k, v, table = cc.paged(lens, hkv, page, rng)
    q = rng.standard_normal((int(cc.starts(lens)[-1]), hq, cc.D)).astype(np.float16)
    args = [dev(a, cuda) for a in (q, k, v, table, cc.starts(lens), np.array([c for _, c in lens], dtype=np.int32))]
    ws = torch.empty(i4lib.paged_gqa_chunk_ws_bytes(), dtype=torch.uint8, device=cuda)
    run = lambda: i4lib.paged_gqa_chunk(*args, window=window, ws=ws)  # noqa: E731
    first = run()
    assert all(torch.equal(run(), first) for _ in range(20))
    side, x = torch.cuda.Stream(), torch.randn((4096, 4096), device=cuda)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(10):
            x = x @ x * 1e-3
    assert all(torch.equal(run(), first) for _ in range(20))
    i4lib.set_option("pdl", 0)
    try:
        assert all(torch.equal(run(), first) for _ in range(3))
    finally:
        i4lib.set_option("pdl", 1)
    torch.cuda.synchronize()
    assert i4lib.device_error() == 0
