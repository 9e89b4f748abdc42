"""Attention of new tokens where its numbers are hard: weights far below the row's largest, scores of any finite size
(needs a B200)."""
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


def test_rows_summed_again_beside_large_scores(i4lib, cuda):
    """Scores of 2^30 and a NaN in the last token's V: the other rows are summed again and still give their largest's V."""
    for n, ctx in ((3, 700), (6, 9000), (300, 1300)):
        lens, q, k, v, table, top = needle_case(n, ctx, 4096.0, seed=n + ctx)
        want = cc.rows_of(v, table[0], ctx, 16)[top, 0].astype(np.float64)
        put(v, table, 0, ctx - 1, np.nan)
        got = call(i4lib, cuda, q, k, v, table, lens)[:-1]
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -10 + 2.0 ** -13) + 2.0 ** -25)
