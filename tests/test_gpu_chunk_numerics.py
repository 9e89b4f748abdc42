"""Attention of new tokens where its numbers are hard: weights far below the row's largest (needs a B200)."""
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
