"""Calls on ragged batches and on the cache's pages that are refused before anything is launched (no GPU needed)."""
import ctypes

import pytest

FAKE = 1 << 20  # an address that is never followed: validation fails first


FIELDS = dict(k="k_pool", v="v_pool", table="page_table", ctx="ctx_len", page="page_size", max_pages="max_pages_per_seq",
              pages="num_pages", stride="qkv_stride", rd="rotary_dim", inter="interleaved")


def status(fn, base, args=None, **change):
    names = [n for n, _ in base]
    values = dict(base, **change)
    assert set(change) <= set(names)
    if args is None:
        return fn(*[values[n] for n in names])
    return fn(ctypes.byref(args(**{FIELDS.get(n, n): v for n, v in values.items()})), None)


ATTN = [("q", FAKE), ("q_stride", 28 * 128), ("k", FAKE), ("v", FAKE), ("table", FAKE), ("q_start", FAKE), ("ctx", FAKE), ("out", FAKE),
        ("T", 10), ("B", 2), ("Hq", 28), ("Hkv", 4), ("D", 128), ("page", 16), ("max_pages", 8), ("pages", 20), ("window", 0),
        ("max_q", 0), ("scale", 0.1), ("ws", FAKE), ("ws_bytes", 1)]


@pytest.mark.parametrize("change,want", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1), (dict(q_start=None), -1), (dict(ctx=None), -1),
    (dict(out=None), -1), (dict(T=0), -1), (dict(B=0), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(max_pages=0), -1),
    (dict(pages=0), -1), (dict(window=-1), -1), (dict(max_q=-1), -1), (dict(D=64), -3), (dict(Hq=30, q_stride=30 * 128), -3),
    (dict(Hq=36, q_stride=36 * 128), -3), (dict(page=4), -3), (dict(page=24), -3), (dict(page=256), -3), (dict(T=(1 << 20) + 1), -3),
    (dict(B=65537), -3), (dict(max_pages=1 << 17), -3), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=float("inf")), -1), (dict(scale=1e21), -1), (dict(q_stride=28 * 128 - 8), -1), (dict(q_stride=28 * 128 + 4), -1), (dict(q=FAKE + 8), -2),
    (dict(k=FAKE + 8), -2), (dict(v=FAKE + 2), -2), (dict(out=FAKE + 8), -2), (dict(table=FAKE + 2), -2), (dict(q_start=FAKE + 1), -2),
    (dict(T=1 << 20, B=65536, Hkv=4096, Hq=4096, q_stride=4096 * 128, max_pages=1 << 16, ws_bytes=1 << 40), -3),
    (dict(ws=None), -1), (dict(), -1), (dict(ws_bytes=1 << 40, ws=FAKE + 16), -2),
])
def test_attention(i4lib, change, want):
    assert status(i4lib.lib().i4_paged_gqa_chunk, ATTN, i4lib.ChunkAttnArgs, **change) == want
    assert i4lib.lib().i4_last_error()


ROPE = [("qkv", FAKE), ("stride", 36 * 128), ("q_start", FAKE), ("ctx", FAKE), ("cs", FAKE), ("max_pos", 100), ("rd", 128), ("inter", 0),
        ("T", 4), ("B", 2), ("Hq", 28), ("Hkv", 4), ("D", 128), ("q_out", FAKE), ("k", FAKE), ("v", FAKE), ("table", FAKE), ("page", 16),
        ("max_pages", 4), ("pages", 8)]


@pytest.mark.parametrize("change,want", [
    (dict(qkv=None), -1), (dict(q_start=None), -1), (dict(ctx=None), -1), (dict(cs=None), -1), (dict(q_out=None), -1), (dict(k=None), -1),
    (dict(v=None), -1), (dict(table=None), -1), (dict(D=64), -3), (dict(rd=0), -3), (dict(rd=24), -3), (dict(rd=144), -3), (dict(T=0), -1),
    (dict(B=0), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(max_pos=0), -1), (dict(page=0), -1), (dict(max_pages=0), -1),
    (dict(pages=0), -1), (dict(Hq=5000, stride=5008 * 128), -1), (dict(stride=36 * 128 - 8), -1), (dict(stride=36 * 128 + 4), -1),
    (dict(qkv=FAKE + 8), -2), (dict(cs=FAKE + 8), -2), (dict(q_out=FAKE + 8), -2), (dict(k=FAKE + 8), -2), (dict(ctx=FAKE + 2), -2),
])
def test_rope_append(i4lib, change, want):
    assert status(i4lib.lib().i4_rope_append_chunk, ROPE, i4lib.RopeChunkArgs, **change) == want


def test_null_arguments(i4lib):
    assert i4lib.lib().i4_rope_append_chunk(None, None) == -1
    assert i4lib.lib().i4_paged_gqa_chunk(None, None) == -1


def test_packed_arguments_are_the_structures(i4lib):
    """The calls pack the header's structures themselves: the same sizes, and every field at its place."""
    for packed, st in ((i4lib._ROPE_CHUNK, i4lib.RopeChunkArgs), (i4lib._CHUNK_ATTN, i4lib.ChunkAttnArgs),
                       (i4lib._CACHE, i4lib.KvCacheDesc)):
        names = [n for n, _ in st._fields_]
        assert packed.size == ctypes.sizeof(st)
        got = st.from_buffer_copy(packed.pack(*range(1, len(names) + 1)))
        assert [getattr(got, n) for n in names] == list(range(1, len(names) + 1))


TABLE = [("cs", FAKE), ("max_pos", 10), ("rd", 128), ("theta", 1e6), ("scaling", 2), ("factor", 4.0), ("original", 1024), ("stream", None)]


@pytest.mark.parametrize("change,want", [
    (dict(cs=None), -1), (dict(max_pos=0), -1), (dict(rd=8), -3), (dict(rd=136), -3), (dict(rd=256), -3), (dict(theta=1.0), -1),
    (dict(theta=float("nan")), -1), (dict(theta=float("inf")), -1), (dict(scaling=3), -1), (dict(scaling=-1), -1), (dict(factor=0.5), -1),
    (dict(factor=float("inf")), -1), (dict(original=0), -1), (dict(cs=FAKE + 8), -2),
])
def test_rope_table(i4lib, change, want):
    assert status(i4lib.lib().i4_rope_table, TABLE, **change) == want


def test_pages(i4lib):
    L = i4lib.lib()
    fake = ctypes.c_void_p(FAKE)
    pools = (ctypes.c_void_p * 2)(FAKE, FAKE)
    holed = (ctypes.c_void_p * 2)(FAKE, None)
    odd = (ctypes.c_void_p * 2)(FAKE, FAKE + 8)

    def desc(**kw):
        d = dict(table=FAKE, ctx=FAKE, refs=FAKE, n=8, width=4, page=16, pages=32)
        d.update(kw)
        return ctypes.byref(i4lib.KvCacheDesc(d["table"], d["ctx"], d["refs"], d["n"], d["width"], d["page"], d["pages"]))

    big = 1 << 30
    for kw, want in ((dict(table=None), -1), (dict(ctx=None), -1), (dict(refs=None), -1), (dict(n=0), -1), (dict(width=0), -1),
                     (dict(page=0), -1), (dict(pages=0), -1), (dict(pages=(1 << 20) + 1), -1), (dict(n=16385), -3),
                     (dict(table=FAKE + 2), -2), (dict(width=1 << 28), -1)):
        assert L.i4_kv_pages_reserve(desc(**kw), fake, fake, 1, None, fake, big, None) == want, kw
        assert L.i4_kv_pages_fork(desc(**kw), pools, 2, 4, 128, fake, fake, 1, None, fake, big, None) == want, kw
        assert L.i4_kv_pages_free(desc(**kw), fake, 1, None) == want, kw
        assert L.i4_kv_pages_compact(desc(**kw), pools, 2, 4, 128, None, fake, big, None) == want, kw
    assert L.i4_kv_pages_reserve(None, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_reserve(desc(), None, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_reserve(desc(), fake, None, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_reserve(desc(), fake, fake, -1, None, fake, big, None) == -1
    assert L.i4_kv_pages_reserve(desc(), fake, fake, 9, None, fake, big, None) == -1   # more requests than sequences
    assert L.i4_kv_pages_reserve(desc(), fake, fake, 1, None, None, big, None) == -1
    assert L.i4_kv_pages_reserve(desc(), fake, fake, 1, None, fake, i4lib.kv_pages_ws_bytes(32, 8) - 1, None) == -1
    assert L.i4_kv_pages_reserve(desc(), fake, fake, 1, None, ctypes.c_void_p(FAKE + 8), big, None) == -2
    assert L.i4_kv_pages_reserve(desc(), None, None, 0, None, fake, big, None) == 0    # nothing asked, nothing launched
    assert L.i4_kv_pages_fork(desc(), pools, 2, 4, 128, None, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), pools, 2, 4, 128, fake, fake, 9, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), None, 2, 4, 128, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), pools, 0, 4, 128, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), holed, 2, 4, 128, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), odd, 2, 4, 128, fake, fake, 1, None, fake, big, None) == -2
    assert L.i4_kv_pages_fork(desc(), pools, 2, 4, 100, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), pools, 2, 0, 128, fake, fake, 1, None, fake, big, None) == -1
    assert L.i4_kv_pages_fork(desc(), pools, 2, 4, 128, None, None, 0, None, fake, big, None) == 0
    assert L.i4_kv_pages_free(desc(), None, 1, None) == -1
    assert L.i4_kv_pages_free(desc(), None, 0, None) == 0
    assert L.i4_kv_pages_copy(pools, 2, 32, 4, 16, 128, None, fake, 1, None) == -1
    assert L.i4_kv_pages_copy(pools, 2, 32, 4, 16, 128, fake, fake, -1, None) == -1
    assert L.i4_kv_pages_copy(pools, 2, 0, 4, 16, 128, fake, fake, 1, None) == -1
    assert L.i4_kv_pages_copy(pools, 2, 32, 4, 16, 128, None, None, 0, None) == 0
    assert L.i4_kv_pages_copy(pools, 2, 32, 4, 16, 128, ctypes.c_void_p(FAKE + 2), fake, 1, None) == -2
    assert L.i4_kv_pages_compact(desc(), pools, 2, 4, 128, None, fake, 16, None) == -1
    assert i4lib.kv_pages_ws_bytes(0, 1) == 0 and i4lib.kv_pages_ws_bytes(1, 0) == 0 and i4lib.kv_pages_ws_bytes(8, 1 << 20) == 0
    assert i4lib.kv_pages_ws_bytes(32, 8) > 0


def test_python_calls_refuse_what_they_could_not_follow(i4lib):
    """Tensors off the current device, of another type or shape, never reach the library."""
    import torch
    f16, i32 = torch.float16, torch.int32
    q, pool = torch.zeros((2, 4, 128), dtype=f16), torch.zeros((3, 2, 16, 128), dtype=f16)
    table, start, ctx = torch.zeros((1, 2), dtype=i32), torch.tensor([0, 2], dtype=i32), torch.tensor([5], dtype=i32)
    cs = torch.zeros((10, 64, 2))
    with pytest.raises(i4lib.I4Error, match="CUDA device"):
        i4lib.paged_gqa_chunk(q, pool, pool, table, start, ctx)
    with pytest.raises(i4lib.I4Error, match="fp16"):
        i4lib.paged_gqa_chunk(q.float(), pool, pool, table, start, ctx)
    with pytest.raises(i4lib.I4Error, match="adjacent"):
        i4lib.paged_gqa_chunk(q.transpose(0, 1), pool, pool, table, start, ctx)
    with pytest.raises(i4lib.I4Error, match="int32"):
        i4lib.paged_gqa_chunk(q, pool, pool, table.long(), start, ctx)
    with pytest.raises(i4lib.I4Error, match="contiguous"):
        i4lib.paged_gqa_chunk(q, pool.transpose(1, 2), pool, table, start, ctx)
    qkv = torch.zeros((2, 8 * 128), dtype=f16)
    with pytest.raises(i4lib.I4Error, match="CUDA device"):
        i4lib.rope_append_chunk(qkv, start, ctx, cs, 4, 2, pool, pool, table)
    with pytest.raises(i4lib.I4Error, match="adjacent"):
        i4lib.rope_append_chunk(qkv.t(), start, ctx, cs, 4, 2, pool, pool, table)
    with pytest.raises(i4lib.I4Error, match="scaling"):
        i4lib.rope_table(10, scaling="other", device="cpu")
    refs, seq = torch.zeros(3, dtype=i32), torch.zeros(1, dtype=i32)
    with pytest.raises(i4lib.I4Error, match="CUDA device"):
        i4lib.kv_pages_fork([pool, pool], table, ctx, refs, seq, seq)
    with pytest.raises(i4lib.I4Error, match="pools"):
        i4lib.kv_pages_copy([], seq, seq)
    with pytest.raises(i4lib.I4Error, match="CUDA device"):
        i4lib.kv_pages_reserve(table, ctx, refs, 16, seq, seq)
    with pytest.raises(i4lib.I4Error, match="int32"):
        i4lib.kv_pages_free(table, ctx.long(), refs, 16, seq)


@pytest.mark.parametrize("change,max_tokens", [
    (dict(page_size=24), 16), (dict(page_size=256), 16), (dict(n_q=9, n_kv=1), 16), (dict(n_q=7, n_kv=2), 16), (dict(head_dim=64), 16),
    (dict(page_size=16, max_pages=65537), 16), (dict(), 0), (dict(), 65536),
])
def test_decoder_over_what_its_calls_do_not_take(i4lib, change, max_tokens):
    """Refused when it is made, not by a call in the middle of a run, whose reservation would stay."""
    from types import SimpleNamespace
    d = dict(dict(page_size=16, n_q=4, n_kv=2, head_dim=128, max_pages=4), **change)
    cache = SimpleNamespace(max_pages=d.pop("max_pages"))
    with pytest.raises(ValueError, match="ChunkedDecoder"):
        i4lib.ChunkedDecoder(SimpleNamespace(shape=SimpleNamespace(**d), device="cpu"), cache, max_tokens)
