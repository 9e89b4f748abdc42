"""Rotary positions of new tokens and their append to the pages against the formula in 64 bits (needs a B200)."""
import numpy as np
import pytest

import chunk_cases as cc
from helpers import dev

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


def table_bound(f, m, max_pos):
    """The table holds fp32 roundings of 64-bit values: half a step of fp32, and 2^-40 for the 64-bit angle of the last
    position (2^-53 of an angle up to 2^17, and the functions' own 2 steps)."""
    return m * (2.0 ** -24 + 2.0 ** -35)


@pytest.mark.parametrize("scaling,factor,original", [("none", 1.0, 0), ("linear", 4.0, 0), ("yarn", 4.0, 32768), ("yarn", 1.0, 4096),
                                                     ("yarn", 16.0, 2048)])
@pytest.mark.parametrize("rd", [16, 64, 96, 128])
def test_table(i4lib, cuda, rd, scaling, factor, original):
    max_pos = 131072
    cs = i4lib.rope_table(max_pos, rd, 1e6, scaling, factor, original).cpu().numpy().astype(np.float64)
    f, m = cc.frequencies(rd, 1e6, scaling, factor, original)
    for p in (0, 1, 2, 1000, 65535, max_pos - 1):
        want = np.stack([m * np.cos(p * f), m * np.sin(p * f)], axis=1)
        assert np.abs(cs[p] - want).max() <= table_bound(f, m, max_pos)


def run(i4, cuda, lens, hq, hkv, page, rd, interleaved, pad=0, seed=0, scaling=("none", 1.0, 0), table=None, pages=None, max_pos=8192,
        stride=0):
    import torch
    rng = np.random.default_rng(seed)
    T = int(cc.starts(lens)[-1]) + pad
    width = (hq + 2 * hkv) * cc.D
    qkv = rng.standard_normal((T, width + stride)).astype(np.float16)
    k, v, own = cc.paged(lens, hkv, page, rng)
    table = own if table is None else table
    cs = i4.rope_table(max_pos, rd, 1e6, *scaling)
    q_out = torch.full((T, hq, cc.D), SENTINEL, dtype=torch.float16, device=cuda)
    tk, tv = dev(k, cuda), dev(v, cuda)
    x = dev(qkv, cuda)[:, :width]
    i4.rope_append_chunk(x, dev(cc.starts(lens), cuda), dev(np.array([c for _, c in lens], dtype=np.int32), cuda), cs, hq, hkv, tk, tv,
                         dev(table, cuda), q_out=q_out, interleaved=interleaved)
    torch.cuda.synchronize()
    assert torch.equal(x, dev(qkv, cuda)[:, :width])
    return qkv[:, :width], (k, v), table, [t.cpu().numpy() for t in (q_out, tk, tv)]


def check(lens, hq, hkv, page, rd, interleaved, scaling, qkv, before, table, got, skip=()):
    """A rotated value is two fp32 products of table entries that are off by 2^-24 m, summed in fp32 and rounded once to
    fp16: half a step of the result (2^-11 of it, 2^-25 where it is subnormal) and 3 * 2^-23 m (|a| + |b|)."""
    f, m = cc.frequencies(rd, 1e6, *scaling)
    s0 = cc.starts(lens)
    want_k, want_v = before[0].copy(), before[1].copy()
    touched = np.zeros(want_k.shape[:3:2], dtype=bool)
    for b, (n, ctx) in enumerate(lens):
        for i in range(n):
            row = qkv[s0[b] + i].reshape(-1, cc.D)
            pos = ctx - n + i
            if (b, i) in skip:
                assert np.all(got[0][s0[b] + i] == SENTINEL)
                continue
            want = cc.rotate(row[:hq + hkv], pos, f, m, interleaved)
            page_id, slot = table[b, pos // page], pos % page
            out = np.concatenate([got[0][s0[b] + i], got[1][page_id, :, slot]]).astype(np.float64)
            x = np.abs(row[:hq + hkv].astype(np.float64))
            bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 3 * 2.0 ** -23 * m * (x + x.max(axis=-1, keepdims=True))
            assert np.all(np.abs(out - want) <= bound)
            assert np.array_equal(out[:, rd:], row[:hq + hkv, rd:].astype(np.float64))
            want_v[page_id, :, slot] = row[hq + hkv:]
            want_k[page_id, :, slot] = got[1][page_id, :, slot]
            touched[page_id, slot] = True
    assert np.array_equal(got[1].view(np.uint16), want_k.view(np.uint16))  # nothing else was written
    assert np.array_equal(got[2].view(np.uint16), want_v.view(np.uint16))
    assert np.all(got[0][s0[-1]:] == SENTINEL)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rd", [16, 32, 48, 64, 96, 112, 128])
def test_layouts(i4lib, cuda, rd, interleaved):
    lens = [(1, 1), (5, 40), (0, 3), (17, 17), (1, 4001)]
    r = run(i4lib, cuda, lens, 7, 1, 16, rd, interleaved, pad=3, seed=rd)
    check(lens, 7, 1, 16, rd, interleaved, ("none", 1.0, 0), *r)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 1), (6, 2), (28, 4), (32, 32), (64, 8), (3, 3)])
def test_head_counts(i4lib, cuda, hq, hkv):
    lens = [(3, 70), (1, 8)]
    for interleaved in (False, True):
        r = run(i4lib, cuda, lens, hq, hkv, 8, 128, interleaved, seed=hq)
        check(lens, hq, hkv, 8, 128, interleaved, ("none", 1.0, 0), *r)


@pytest.mark.parametrize("scaling", [("linear", 4.0, 0), ("yarn", 4.0, 1024)])
def test_scaled_positions_and_strided_rows(i4lib, cuda, scaling):
    lens = [(9, 5000), (200, 300)]
    r = run(i4lib, cuda, lens, 4, 2, 64, 64, True, seed=1, scaling=scaling, stride=24)
    check(lens, 4, 2, 64, 64, True, scaling, *r)


@pytest.mark.parametrize("n_seq", [31, 32, 33, 64, 1030])
def test_many_sequences(i4lib, cuda, n_seq):
    rng = np.random.default_rng(n_seq)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 3, n_seq), rng.integers(0, 30, n_seq))]
    r = run(i4lib, cuda, lens, 2, 1, 8, 128, False, seed=n_seq, pad=1)
    check(lens, 2, 1, 8, 128, False, ("none", 1.0, 0), *r)


def test_tokens_without_a_place_are_skipped(i4lib, cuda):
    """Positions below zero, behind the table of angles and behind the page-table row."""
    lens = [(4, 2), (3, 33), (2, 61)]  # positions -2..1, 30..32 (the row holds 32), 59..60 (60 angles)
    rng = np.random.default_rng(0)
    table = np.full((3, 8), -1, dtype=np.int32)
    table[0, 0], table[1, :4], table[2] = 0, [1, 2, 3, 4], range(5, 13)
    table[1, 4:] = -1
    lens_alloc = [(4, 8), (3, 32), (2, 64)]
    import torch
    k, v, _ = cc.paged(lens_alloc, 1, 8, rng)
    qkv = rng.standard_normal((9, 4 * 128)).astype(np.float16)
    cs = i4lib.rope_table(60, 128, 1e6)
    q_out = torch.full((9, 2, 128), SENTINEL, dtype=torch.float16, device=cuda)
    tk, tv = dev(k, cuda), dev(v, cuda)
    i4lib.rope_append_chunk(dev(qkv, cuda), dev(cc.starts(lens), cuda), dev(np.array([2, 33, 61], dtype=np.int32), cuda), cs, 2, 1, tk,
                            tv, dev(table, cuda), q_out=q_out)
    got = [t.cpu().numpy() for t in (q_out, tk, tv)]
    assert np.all(got[0][[0, 1, 8]] == SENTINEL) and not np.any(got[0][[2, 3, 4, 5, 6, 7]] == SENTINEL)
    # position 32 of sequence 1 has the page id -1: its q is written, its K/V nowhere
    changed = np.argwhere(np.any(got[2].view(np.uint16) != v.view(np.uint16), axis=(1, 3)))
    assert {tuple(x) for x in changed} == {(0, 0), (0, 1), (4, 6), (4, 7), (12, 3)}


def test_angles_of_far_positions(i4lib, cuda):
    """Positions near 2^17, where an fp32 angle would be off by more than the fp16 step."""
    lens = [(2, 131072)]
    r = run(i4lib, cuda, lens, 1, 1, 128, 128, False, seed=2, max_pos=131072)
    check(lens, 1, 1, 128, 128, False, ("none", 1.0, 0), *r)


def test_same_as_the_single_token_call(i4lib, cuda):
    """rotate-half over the whole head at one token a sequence: the same bits as rope_kv_append but where a rounding of the
    angle's cosine crosses a step."""
    import torch
    lens = [(1, c) for c in (1, 9, 200, 4000)]
    qkv, before, table, got = run(i4lib, cuda, lens, 7, 1, 16, 128, False, seed=3)
    x = dev(qkv, cuda)
    tk, tv = dev(before[0], cuda), dev(before[1], cuda)
    i4lib.rope_kv_append(x, dev(np.array([c - 1 for _, c in lens], dtype=np.int32), cuda), 7, 1, 1e6, tk, tv, dev(table, cuda))
    assert np.array_equal(tv.cpu().numpy().view(np.uint16), got[2].view(np.uint16))
    for a, b in ((x.cpu().numpy()[:, :7 * 128].reshape(4, 7, 128), got[0]), (np.nan_to_num(tk.cpu().numpy()), np.nan_to_num(got[1]))):
        a, b = a.astype(np.float64), b.astype(np.float64)
        assert np.all(np.abs(a - b) <= 2.0 ** -10 * np.maximum(np.abs(a), np.abs(b)) + 2.0 ** -20 * 8)


def test_captured_call_follows_the_lengths(i4lib, cuda):
    import torch
    hq, hkv, page = 3, 1, 8
    alloc = [(10, 90), (10, 40)]
    rng = np.random.default_rng(5)
    k, v, table = cc.paged(alloc, hkv, page, rng)
    qkv = rng.standard_normal((20, 5 * 128)).astype(np.float16)
    cs = i4lib.rope_table(128, 128, 1e6)
    x, tt, tk, tv = (dev(a, cuda) for a in (qkv, table, k, v))
    start = torch.tensor([0, 10, 20], dtype=torch.int32, device=cuda)
    ctx = torch.tensor([90, 40], dtype=torch.int32, device=cuda)
    out = torch.full((20, hq, 128), SENTINEL, dtype=torch.float16, device=cuda)
    call = lambda: i4lib.rope_append_chunk(x, start, ctx, cs, hq, hkv, tk, tv, tt, q_out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in (alloc, [(1, 5), (2, 40)], [(0, 0), (20, 40)]):
        start.copy_(torch.from_numpy(cc.starts(lens)))
        ctx.copy_(torch.tensor([c for _, c in lens], dtype=torch.int32))
        out.fill_(SENTINEL)
        tk.copy_(dev(k, cuda))
        tv.copy_(dev(v, cuda))
        g.replay()
        torch.cuda.synchronize()
        check(lens, hq, hkv, page, 128, False, ("none", 1.0, 0), qkv, (k, v), table, [t.cpu().numpy() for t in (out, tk, tv)])
