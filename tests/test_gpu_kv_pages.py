"""Copying, reserving, forking, freeing and compacting pages against plain Python (needs a B200); every comparison is of bits."""
import ctypes

import numpy as np
import pytest

import chunk_cases as cc
from helpers import dev

pytestmark = pytest.mark.gpu


class Both:
    """The device's cache beside the model's."""

    def __init__(self, i4, cuda, n_seqs, max_pages, page, num_pages, n_pools=2, hkv=1, d=16, seed=0):
        rng = np.random.default_rng(seed)
        pools = rng.integers(0, 2 ** 16, size=(n_pools, num_pages, hkv, page, d)).astype(np.uint16)
        self.model = cc.PagesModel(np.full((n_seqs, max_pages), -1, dtype=np.int32), np.zeros(n_seqs, dtype=np.int32),
                                   np.zeros(num_pages, dtype=np.int32), pools, page)
        self.i4, self.cuda, self.page = i4, cuda, page
        self.pools = [dev(p.view(np.float16), cuda) for p in pools]
        self.table, self.ctx, self.refs = (dev(a, cuda) for a in (self.model.table, self.model.ctx, self.model.refs))

    def ints(self, v):
        return dev(np.asarray(v, dtype=np.int32), self.cuda)

    def upload(self):
        self.table.copy_(dev(self.model.table, self.cuda))
        self.ctx.copy_(dev(self.model.ctx, self.cuda))
        self.refs.copy_(dev(self.model.refs, self.cuda))

    def reserve(self, seqs, add):
        got = self.i4.kv_pages_reserve(self.table, self.ctx, self.refs, self.page, self.ints(seqs), self.ints(add))
        want = self.model.reserve(seqs, add)
        assert got.cpu().tolist() == want
        self.same()
        return want

    def fork(self, src, dst):
        got = self.i4.kv_pages_fork(self.pools, self.table, self.ctx, self.refs, self.ints(src), self.ints(dst))
        want = self.model.fork(src, dst)
        assert got.cpu().tolist() == want
        self.same()
        return want

    def free(self, seqs):
        self.i4.kv_pages_free(self.table, self.ctx, self.refs, self.page, self.ints(seqs))
        for s in set(seqs):
            if 0 <= s < len(self.model.ctx) and self.model.ctx[s] > 0:
                self.model.release(s)
        self.same()

    def compact(self):
        got = self.i4.kv_pages_compact(self.pools, self.table, self.ctx, self.refs)
        want = self.model.compact()
        assert int(got.item()) == want
        self.same()
        return want

    def same(self):
        assert np.array_equal(self.table.cpu().numpy(), self.model.table)
        assert np.array_equal(self.ctx.cpu().numpy(), self.model.ctx)
        assert np.array_equal(self.refs.cpu().numpy(), self.model.refs)
        for a, b in zip(self.pools, self.model.pools):
            assert np.array_equal(a.cpu().numpy().view(np.uint16), b)


def test_reserve(i4lib, cuda):
    c = Both(i4lib, cuda, 8, 6, 8, 12)
    assert c.reserve([3, 0], [9, 8]) == [0, 0]
    assert c.reserve([0, 1, 3], [1, 0, 6]) == [0, 0, 0]
    assert c.reserve([2, 2, -1, 8, 1, 0, 4], [5, 5, 1, 1, -1, 48, 2 ** 31 - 1]) == [0, 2, 2, 2, 2, 2, 2]
    # 12 pages, 6 held: the second request does not fit, nor does the third that needs a page; the fourth needs none
    assert c.reserve([1, 4, 3, 2], [40, 17, 2, 3]) == [0, 1, 1, 0]


def test_reserve_takes_the_last_page(i4lib, cuda):
    c = Both(i4lib, cuda, 2, 8, 8, 4)
    assert c.reserve([0, 1], [24, 8]) == [0, 0]
    assert c.reserve([0, 1], [1, 0]) == [1, 0]
    c.free([1])
    assert c.reserve([0], [8]) == [0]


@pytest.mark.parametrize("page", [8, 16, 5])
@pytest.mark.parametrize("ctx", [1, 4, 5, 8, 16, 17, 39, 40])
def test_fork(i4lib, cuda, page, ctx):
    c = Both(i4lib, cuda, 8, 10, page, 64, n_pools=3, hkv=2, d=128)
    c.reserve([0, 1, 5], [7, ctx, 3])
    assert c.fork([1, 1, 0], [2, 5, 7]) == [0, 0, 0]
    assert c.fork([1, 1], [2, 5]) == [0, 0]  # again: the copies are given back and made anew
    c.free([1])
    assert c.fork([2, 7], [1, 3]) == [0, 0]
    c.reserve([1, 2, 5], [9, 2, 1])


def test_fork_refusals(i4lib, cuda):
    c = Both(i4lib, cuda, 8, 4, 8, 12)
    c.reserve([0, 1], [12, 9])
    #             ok  dst again  src outside  dst outside  src outside  src is a dst  src == dst
    assert c.fork([0, 0, 9, 0, -1, 3, 2], [3, 3, 4, 8, 5, 6, 2]) == [0, 2, 2, 2, 2, 2, 2]
    assert c.fork([1, 0], [0, 4]) == [0, 2]  # 0 becomes a continuation of 1, so 4 cannot continue 0 in the same call


def test_fork_without_a_free_page(i4lib, cuda):
    c = Both(i4lib, cuda, 6, 4, 8, 5)
    c.reserve([0, 1, 4], [12, 9, 8])  # all five pages
    # 4 gives its page back to the first fork; the second finds none and stays empty; the third needs none
    assert c.fork([0, 1], [4, 2]) == [0, 1]
    c.free([0])
    assert c.fork([1, 4], [2, 3]) == [0, 1]


def test_empty_and_unheld_sequences(i4lib, cuda):
    c = Both(i4lib, cuda, 4, 3, 8, 6)
    assert c.fork([0], [1]) == [0]
    c.free([0, 1, 2, 3, 3])
    assert c.compact() == 0
    c.reserve([2], [3])
    assert c.fork([0], [2]) == [0]  # an empty source empties its target
    assert c.compact() == 0


def test_free_twice_and_outside(i4lib, cuda):
    c = Both(i4lib, cuda, 4, 3, 8, 8)
    c.reserve([0, 1, 2], [20, 16, 1])
    c.fork([1], [3])
    c.free([1, 1, -1, 4, 100, 0])
    c.free([3, 2])
    assert int(c.refs.sum().item()) == 0


@pytest.mark.parametrize("num_pages", [1, 3, 40, 1025, 4096, 4097, 9000])
def test_compact(i4lib, cuda, num_pages):
    c = Both(i4lib, cuda, 9, 64, 8, num_pages, seed=num_pages)
    rng = np.random.default_rng(num_pages)
    ids = rng.permutation(num_pages)[:max(1, min(num_pages // 2, 300))]
    at = 0
    for s in range(9):  # pages anywhere in the pools, some held by two sequences
        n = min(int(rng.integers(0, 40)), len(ids) - at)
        c.model.table[s, :n] = ids[at:at + n]
        c.model.ctx[s] = max(0, n * 8 - int(rng.integers(0, 8))) if n else 0
        c.model.refs[ids[at:at + n]] += 1
        at += n
    c.model.table[8, :2] = c.model.table[0, :2]
    if c.model.ctx[0] >= 16 and c.model.ctx[8] == 0:
        c.model.ctx[8] = 16
        c.model.refs[c.model.table[8, :2]] += 1
    else:
        c.model.table[8, :2] = -1
        for p in c.model.table[8, 2:c.model.held(8)]:
            c.model.refs[p] -= 1
        c.model.refs[:] = 0
        c.model.ctx[8] = 0
        for s in range(8):
            c.model.refs[c.model.table[s, :c.model.held(s)]] += 1
    c.upload()
    n = c.compact()
    assert n == int((c.model.refs > 0).sum()) and np.all(c.model.refs[:n] > 0)
    assert c.compact() == n  # nothing left to move


def test_copy(i4lib, cuda):
    import torch
    rng = np.random.default_rng(1)
    for n_pools, hkv, page, d in ((1, 1, 8, 8), (3, 4, 16, 128), (300, 1, 8, 8), (2, 2, 5, 24)):
        host = rng.integers(0, 2 ** 16, size=(n_pools, 12, hkv, page, d)).astype(np.uint16)
        pools = [dev(p.view(np.float16), cuda) for p in host]
        src, dst = [0, 3, 5, -1, 7, 12, 8], [1, 4, 5, 6, 12, 9, 10]
        i4lib.kv_pages_copy(pools, *(dev(np.array(x, dtype=np.int32), cuda) for x in (src, dst)))
        for a, b in zip(src, dst):
            if 0 <= a < 12 and 0 <= b < 12:
                host[:, b] = host[:, a]
        for a, b in zip(pools, host):
            assert np.array_equal(a.cpu().numpy().view(np.uint16), b)
    i4lib.kv_pages_copy(pools, torch.empty(0, dtype=torch.int32, device=cuda), torch.empty(0, dtype=torch.int32, device=cuda))


def test_more_pools_than_one_launch_takes(i4lib, cuda):
    c = Both(i4lib, cuda, 3, 2, 8, 8, n_pools=300, d=8)
    c.reserve([0], [11])
    c.reserve([1], [5])
    c.fork([0], [2])
    c.free([0])
    c.compact()


@pytest.mark.parametrize("seed", range(4))
def test_a_life_of_a_cache(i4lib, cuda, seed):
    rng = np.random.default_rng(seed)
    c = Both(i4lib, cuda, 40, 12, 8, 150, seed=seed)
    for _ in range(30):
        op = rng.integers(0, 5)
        if op <= 1:
            seqs = rng.permutation(40)[:rng.integers(1, 12)].tolist()
            c.reserve(seqs, rng.integers(0, 30, size=len(seqs)).tolist())
        elif op == 2:
            pick = rng.permutation(40)[:rng.integers(2, 20)].tolist()
            src = [pick[0] if rng.random() < 0.5 else pick[1]] * (len(pick) - 2)
            c.fork(src, pick[2:])
        elif op == 3:
            c.free(rng.permutation(40)[:rng.integers(1, 8)].tolist())
        else:
            c.compact()
        assert c.model.refs.min() >= 0


@pytest.mark.parametrize("n_seqs", [1025, 13000])
def test_many_sequences(i4lib, cuda, n_seqs):
    c = Both(i4lib, cuda, n_seqs, 2, 8, 2 * n_seqs + 7, n_pools=1, d=8)
    c.reserve(list(range(n_seqs // 2)), [3 + i % 11 for i in range(n_seqs // 2)])
    m = n_seqs // 2
    assert set(c.fork(list(range(m)), list(range(m, 2 * m)))) == {0}
    c.free(list(range(0, n_seqs, 3)))
    c.compact()


@pytest.mark.parametrize("num_pages", [12000, 52000])
def test_fork_in_a_large_pool(i4lib, cuda, num_pages):
    """More page counts than fit beside the sequences in 48 KB, and in the plan's shared memory at all."""
    c = Both(i4lib, cuda, 30, 20, 8, num_pages, n_pools=1, d=8)
    c.model.refs[:num_pages - 40] = 1  # held by somebody else: the free pages are the last
    c.upload()
    assert c.reserve([0, 1], [150, 33]) == [0, 0]
    assert c.fork([0, 0, 1, 0], [2, 3, 4, 5]) == [0, 0, 0, 0]
    assert c.fork([0, 1], [5, 3]) == [0, 0]
    c.free([0, 3])


def test_captured_operations(i4lib, cuda):
    """Reserve, fork and free in one graph, replayed: every replay acts on the cache as it is."""
    import torch
    c = Both(i4lib, cuda, 4, 8, 8, 40)
    c.reserve([0], [13])
    seq0, seq1, one = c.ints([0]), c.ints([1]), c.ints([3])
    st = [torch.zeros(1, dtype=torch.int32, device=cuda) for _ in range(2)]
    ws = torch.empty(i4lib.kv_pages_ws_bytes(40, 4), dtype=torch.uint8, device=cuda)

    def step():
        i4lib.kv_pages_reserve(c.table, c.ctx, c.refs, 8, seq0, one, status=st[0], ws=ws)
        i4lib.kv_pages_fork(c.pools, c.table, c.ctx, c.refs, seq0, seq1, status=st[1], ws=ws)

    step()
    c.model.reserve([0], [3])
    c.model.fork([0], [1])
    c.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(6):
        g.replay()
        c.model.reserve([0], [3])
        c.model.fork([0], [1])
        c.same()


def test_two_threads_with_caches_of_different_sizes(i4lib, cuda):
    """Each thread has its own cache, workspace and stream. The plans of both need more shared memory than a kernel has without
    asking, one three times the other's. The calls follow each other as fast as a host can make them, so that they meet."""
    import threading
    import torch
    errors, both = [], threading.Barrier(2)

    def work(c, num_pages):
        stream = torch.cuda.Stream()
        ws = torch.empty(i4lib.kv_pages_ws_bytes(num_pages, 30), dtype=torch.uint8, device=cuda)
        src, dst, status = c.ints([0, 0]), c.ints([1, 2]), c.ints([7, 7])
        desc = i4lib.KvCacheDesc(c.table.data_ptr(), c.ctx.data_ptr(), c.refs.data_ptr(), 30, 20, 8, num_pages)
        pools = (ctypes.c_void_p * 1)(c.pools[0].data_ptr())
        fork = i4lib.lib().i4_kv_pages_fork
        args = (ctypes.byref(desc), pools, 1, 1, 8, src.data_ptr(), dst.data_ptr(), 2, status.data_ptr(), ws.data_ptr(), ws.numel(),
                stream.cuda_stream)
        torch.cuda.synchronize()
        both.wait()
        for _ in range(4000):
            st = fork(*args)
            if st:
                errors.append((num_pages, st, i4lib.lib().i4_last_error()))
                return

    caches = [Both(i4lib, cuda, 30, 20, 8, n, n_pools=1, d=8) for n in (13000, 40000)]
    for c in caches:
        c.reserve([0], [13])
    threads = [threading.Thread(target=work, args=(c, len(c.model.refs))) for c in caches]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c in caches:
        c.model.fork([0, 0], [1, 2])
        c.same()


@pytest.mark.parametrize("calls", ["copy", "fork", "compact"])
def test_pools_of_different_layouts_are_refused(i4lib, cuda, calls):
    """The same number of values, but other pages, heads or rows: one call cannot move both."""
    import torch
    c = Both(i4lib, cuda, 4, 3, 8, 6, n_pools=2, hkv=2, d=16)
    c.reserve([0], [11])
    for shape in ((6, 1, 8, 32), (6, 4, 4, 16), (12, 1, 8, 16), (6, 2, 16, 8)):
        pools = [c.pools[0], torch.zeros(shape, dtype=torch.float16, device=cuda)]
        with pytest.raises(i4lib.I4Error, match="one shape"):
            if calls == "copy":
                i4lib.kv_pages_copy(pools, c.ints([0]), c.ints([5]))
            elif calls == "fork":
                i4lib.kv_pages_fork(pools, c.table, c.ctx, c.refs, c.ints([0]), c.ints([1]))
            else:
                i4lib.kv_pages_compact(pools, c.table, c.ctx, c.refs)
    c.same()


def test_pages_that_the_caller_counts_itself(i4lib, cuda):
    """Held out of the cache at the lowest ids they are never handed out, and compaction leaves them where they are."""
    c = Both(i4lib, cuda, 4, 6, 8, 30)
    c.model.refs[:3] = 1
    c.upload()
    before = [p[:3].copy() for p in c.model.pools]
    c.reserve([0, 1, 2], [20, 30, 9])
    c.fork([1], [3])
    c.free([0, 1])
    assert c.compact() == 3 + 2 + 4
    c.free([2, 3])
    assert c.compact() == 3
    for p, b in zip(c.pools, before):
        assert np.array_equal(p[:3].cpu().numpy().view(np.uint16), b)


def test_a_life_without_early_launches(i4lib, cuda):
    i4lib.set_option("pdl", 0)
    try:
        test_a_life_of_a_cache(i4lib, cuda, 9)
        test_captured_operations(i4lib, cuda)
    finally:
        i4lib.set_option("pdl", 1)
