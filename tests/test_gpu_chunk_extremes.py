"""The calls on chunks and pages at the ends of their ranges, and captured before anything was called (needs a B200)."""
import os
import subprocess
import sys

import numpy as np
import pytest

import chunk_cases as cc
from conftest import ROOT
from helpers import dev

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


def attend(i4, cuda, q, k, v, table, lens, page, pad=0, **kw):
    """The call's rows against the bound of cc.attention; `pad` rows behind the last sequence are left alone."""
    import torch
    out = torch.full((q.shape[0], *q.shape[1:]), SENTINEL, dtype=torch.float16, device=cuda)
    i4.paged_gqa_chunk(dev(q, cuda), dev(k, cuda), dev(v, cuda), dev(table, cuda), dev(cc.starts(lens), cuda),
                       dev(np.array([c for _, c in lens], dtype=np.int32), cuda), out=out, **kw)
    torch.cuda.synchronize()
    assert i4.device_error() == 0
    n = q.shape[0] - pad
    want, bound = cc.attention(q[:n], k, v, table, lens, page)
    got = out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got[:n] - want) <= bound)
    assert np.all(got[n:] == SENTINEL)


@pytest.mark.parametrize("max_q", [0, 2])
def test_the_most_sequences(i4lib, cuda, max_q):
    rng = np.random.default_rng(1)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 3, 65536), rng.integers(0, 9, 65536))]
    k, v, table = cc.paged(lens, 1, 8, rng)
    q = rng.standard_normal((int(cc.starts(lens)[-1]) + 5, 1, cc.D)).astype(np.float16)
    attend(i4lib, cuda, q, k, v, table, lens, 8, pad=5, max_q=max_q)


def test_the_most_kv_heads(i4lib, cuda):
    rng = np.random.default_rng(2)
    lens = [(2, 9), (1, 3)]
    k, v, table = cc.paged(lens, 4096, 8, rng)
    q = rng.standard_normal((3, 4096, cc.D)).astype(np.float16)
    attend(i4lib, cuda, q, k, v, table, lens, 8)


def test_the_most_tokens(i4lib, cuda):
    """2^20 new tokens, prompts of 2^16 beside each other; rows here and there against 64 bits."""
    import torch
    T, n_seq, page = 1 << 20, 16, 128
    each = T // n_seq
    gen = torch.Generator(device=cuda).manual_seed(3)
    q = torch.randn((T, 1, 128), generator=gen, device=cuda, dtype=torch.float16)
    k, v = (torch.randn((T // page, 1, page, 128), generator=gen, device=cuda, dtype=torch.float16) for _ in range(2))
    v += 1
    perm = torch.randperm(T // page, generator=gen, device=cuda)
    table = perm.to(torch.int32).view(n_seq, -1).contiguous()
    start = torch.arange(0, T + 1, each, dtype=torch.int32, device=cuda)
    ctx = torch.full((n_seq,), each, dtype=torch.int32, device=cuda)
    got = i4lib.paged_gqa_chunk(q, k, v, table, start, ctx)
    assert i4lib.device_error() == 0 and bool(torch.isfinite(got).all())
    kk, vv = (t[perm][:, 0].reshape(n_seq, each, 128).double() for t in (k, v))
    rng = np.random.default_rng(4)
    for t in [0, 1, each - 1, each, T - 1, *rng.integers(0, T, 60).tolist()]:
        b, i = divmod(t, each)
        s = kk[b, :i + 1] @ q[t, 0].double() / np.sqrt(128)
        p = torch.softmax(s, dim=0)
        want, a = p @ vv[b, :i + 1], p @ vv[b, :i + 1].abs()
        e = 128 * 2.0 ** -23 / np.sqrt(128) * (kk[b, :i + 1].abs() @ q[t, 0].double().abs()).max()
        tiny = p.max() * 2.0 ** -32 * vv[b, :i + 1].abs().sum(0)
        bound = 2.0 ** -11 * (a + want.abs()) + 2 * e * a + 2 * 640 * 2.0 ** -23 * a + tiny + 2.0 ** -25
        assert bool(((got[t, 0].double() - want).abs() <= bound).all()), t


def test_rows_summed_again_over_long_contexts(i4lib, cuda):
    """A NaN in the last token's V makes 15 of 16 tokens be summed again over 2^19 positions, 32 rows a warp, in two whole units a
    CTA: longer than any other wait of the kernel may take, and the second unit's roles wait for it."""
    import torch
    ctx, page, n_seq, n, heads = 1 << 19, 128, 296, 16, 8
    gen = torch.Generator(device=cuda).manual_seed(7)
    k, v = (torch.randn((ctx // page, 1, page, 128), generator=gen, device=cuda, dtype=torch.float16) for _ in range(2))
    v += 1
    q = torch.randn((n_seq * n, heads, 128), generator=gen, device=cuda, dtype=torch.float16)
    perm = torch.randperm(ctx // page, generator=gen, device=cuda)
    v[perm[-1], 0, -1] = float("nan")
    table = perm.to(torch.int32)[None].repeat(n_seq, 1).contiguous()
    start = torch.arange(0, n_seq * n + 1, n, dtype=torch.int32, device=cuda)
    lens = torch.full((n_seq,), ctx, dtype=torch.int32, device=cuda)
    got = i4lib.paged_gqa_chunk(q, k, v, table, start, lens, max_q=n).view(n_seq, n, heads, 128).double()
    assert i4lib.device_error() == 0
    assert bool(torch.isnan(got[:, -1]).all()) and bool(torch.isfinite(got[:, :-1]).all())
    kk, vv = (t[perm][:, 0].reshape(-1, 128).double() for t in (k, v))
    for b, i in ((0, 0), (0, 14), (100, 7), (147, 3), (148, 14), (295, 0), (295, 14)):
        sees = ctx - n + 1 + i
        s = q[b * n + i].double() @ kk[:sees].T / np.sqrt(128)
        p = torch.softmax(s, dim=1)
        want, a = p @ vv[:sees], p @ vv[:sees].abs()
        e = 128 * 2.0 ** -23 / np.sqrt(128) * (q[b * n + i].double().abs() @ kk[:sees].abs().T).amax(dim=1, keepdim=True)
        # the result's rounding and exp's approximation, its scores, fp32 sums of 2^14 trips of 32 (of P V and of P)
        bound = 2.0 ** -11 * want.abs() + 2.0 ** -20 * a + 2 * e * a + 2 * (2 ** 14 + 32) * 2.0 ** -23 * a + 2.0 ** -25
        assert bool((want.abs() > 8 * bound).all())
        assert bool(((got[b, i] - want).abs() <= bound).all()), (b, i)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_append_with_the_most_heads(i4lib, cuda, interleaved):
    import torch
    heads, lens, page = 4096, [(2, 9), (1, 3)], 8
    rng = np.random.default_rng(5)
    k, v, table = cc.paged(lens, heads, page, rng)
    qkv = rng.standard_normal((3, 3 * heads * cc.D)).astype(np.float16)
    cs = i4lib.rope_table(16, 128, 1e6)
    tk, tv = dev(k, cuda), dev(v, cuda)
    got = i4lib.rope_append_chunk(dev(qkv, cuda), dev(cc.starts(lens), cuda), dev(np.array([9, 3], dtype=np.int32), cuda), cs, heads, heads,
                                  tk, tv, dev(table, cuda), interleaved=interleaved).cpu().numpy()
    torch.cuda.synchronize()
    f, m = cc.frequencies(128, 1e6)
    x = qkv.reshape(3, 3 * heads, cc.D)
    for t, (b, pos) in enumerate(((0, 7), (0, 8), (1, 2))):
        y = cc.rotate(x[t, :2 * heads], pos, f, m, interleaved)
        # a product and a sum in fp32 of values below 2^3 with angles off by 2^-24, then fp16: half a step and 2^-20
        page_of = table[b, pos // page]
        for have, want in ((got[t], y[:heads]), (tk[page_of, :, pos % page].cpu().numpy(), y[heads:])):
            assert np.all(np.abs(have.astype(np.float64) - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -20)
        assert np.array_equal(tv[page_of, :, pos % page].cpu().numpy().view(np.uint16), x[t, 2 * heads:].view(np.uint16))


def test_the_largest_cache(i4lib, cuda):
    """2^20 pages and 16384 sequences: counts by numpy, pages by their ids (each page holds its own)."""
    import torch
    pages, n = 1 << 20, 16384
    i32 = dict(dtype=torch.int32, device=cuda)
    ids = torch.arange(pages, **i32)
    pool = torch.zeros((pages, 1, 1, 8), dtype=torch.float16, device=cuda)
    pool.view(torch.int32).view(pages, 4)[:, 0] = ids
    table, ctx, refs = torch.full((n, 60), -1, **i32), torch.zeros(n, **i32), torch.zeros(pages, **i32)
    ws = torch.empty(i4lib.kv_pages_ws_bytes(pages, n), dtype=torch.uint8, device=cuda)
    rng = np.random.default_rng(6)
    order, add = rng.permutation(n).astype(np.int32), rng.integers(0, 61, n).astype(np.int32)
    st = i4lib.kv_pages_reserve(table, ctx, refs, 1, dev(order, cuda), dev(add, cuda), ws=ws)
    assert int(st.abs().sum().item()) == 0
    want, at = np.full((n, 60), -1, dtype=np.int32), 0
    for s, a in zip(order, add):
        want[s, :a] = np.arange(at, at + a)
        at += a
    assert np.array_equal(table.cpu().numpy(), want) and int(refs.sum().item()) == at
    # one in three goes, the last sixth continues others, then the pages close up
    gone = order[::3]
    i4lib.kv_pages_free(table, ctx, refs, 1, dev(gone, cuda))
    want[gone] = -1
    left = np.setdiff1d(order, gone)
    src, dst = left[:2000], gone[:2000]
    st = i4lib.kv_pages_fork([pool], table, ctx, refs, dev(src, cuda), dev(dst, cuda), ws=ws)
    assert int(st.abs().sum().item()) == 0
    want[dst] = want[src]
    assert np.array_equal(table.cpu().numpy(), want)
    count = np.bincount(want[want >= 0], minlength=pages)
    assert np.array_equal(refs.cpu().numpy(), count)
    live = int(i4lib.kv_pages_compact([pool], table, ctx, refs, ws=ws).item())
    assert live == int((count > 0).sum())
    held, moved = pool.view(torch.int32).view(pages, 4)[:, 0].cpu().numpy(), table.cpu().numpy()
    assert np.array_equal(moved >= 0, want >= 0) and moved.max() < live
    assert np.array_equal(held[moved[moved >= 0]], want[want >= 0])  # every entry's page holds what it held
    assert np.array_equal(refs.cpu().numpy(), np.bincount(moved[moved >= 0], minlength=pages))


def test_lists_of_no_entries(i4lib, cuda):
    import torch
    i32 = dict(dtype=torch.int32, device=cuda)
    table, ctx, refs, none = torch.full((3, 4), -1, **i32), torch.zeros(3, **i32), torch.zeros(9, **i32), torch.empty(0, **i32)
    pool = torch.zeros((9, 1, 8, 8), dtype=torch.float16, device=cuda)
    assert i4lib.kv_pages_reserve(table, ctx, refs, 8, none, none).numel() == 0
    assert i4lib.kv_pages_fork([pool], table, ctx, refs, none, none).numel() == 0
    i4lib.kv_pages_free(table, ctx, refs, 8, none)
    i4lib.kv_pages_copy([pool], none, none)


FIRST_CALL = """
import numpy as np, torch
import int4_weight_only_02_b200 as i4
torch.cuda.init()
i32, f16 = dict(dtype=torch.int32, device="cuda"), dict(dtype=torch.float16, device="cuda")
pools = [torch.zeros((24, 1, 8, 128), **f16) for _ in range(2)]
table, ctx, refs = torch.full((3, 40), -1, **i32), torch.zeros(3, **i32), torch.zeros(24, **i32)
ws = torch.empty(i4.kv_pages_ws_bytes(24, 3), dtype=torch.uint8, device="cuda")
attn_ws = torch.empty(i4.paged_gqa_chunk_ws_bytes(), dtype=torch.uint8, device="cuda")
seq, add, one, start = torch.tensor([0], **i32), torch.tensor([40], **i32), torch.tensor([1], **i32), torch.tensor([0, 40, 40, 40], **i32)
angle = torch.arange(320, dtype=torch.float64, device="cuda")[:, None] * 1e6 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
cs = torch.stack([angle.cos(), angle.sin()], dim=2).float().contiguous()
qkv = torch.randn((40, 3 * 128), **f16)
q, out, status, live = torch.zeros((40, 1, 128), **f16), torch.zeros((40, 1, 128), **f16), torch.zeros(2, **i32), torch.zeros(1, **i32)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    made = i4.rope_table(320, 128, 1e6)
    i4.kv_pages_reserve(table, ctx, refs, 8, seq, add, status=status[:1], ws=ws)
    i4.rope_append_chunk(qkv, start, ctx, made, 1, 1, *pools, table, q_out=q)
    i4.paged_gqa_chunk(q, *pools, table, start, ctx, out=out, ws=attn_ws)
    i4.kv_pages_fork(pools, table, ctx, refs, seq, one, status=status[1:], ws=ws)
    i4.kv_pages_free(table, ctx, refs, 8, seq)
    i4.kv_pages_compact(pools, table, ctx, refs, n_live=live, ws=ws)
    i4.kv_pages_copy(pools, seq, one + 20)
g.replay()
torch.cuda.synchronize()
assert i4.device_error() == 0
assert status.tolist() == [0, 0] and ctx.tolist() == [0, 40, 0] and live.item() == 5, (status, ctx, live)
assert (made - cs).abs().max() < 1e-6
v = qkv[:, 256:].double()
k = qkv[:, 128:256].double()
def turn(x):
    a, b = x[:, :64], x[:, 64:]
    c, s = angle[:40].cos(), angle[:40].sin()
    return torch.cat([a * c - b * s, b * c + a * s], dim=1)
s = (turn(qkv[:, :128].double()) @ turn(k).T) / 128 ** 0.5
s = s.masked_fill(torch.ones_like(s).triu(1).bool(), -float("inf"))
want = torch.softmax(s, dim=1) @ v
assert (out[:, 0].double() - want).abs().max() < 0.02 and out.abs().max() > 0.5
print("captured first")
"""


def test_captured_before_anything_was_called(i4lib, cuda):
    """A process whose first call of every kind is inside a capture: nothing is set up then that a capture does not take."""
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]
