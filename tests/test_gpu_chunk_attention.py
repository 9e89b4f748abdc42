"""Attention of new tokens over the pages against the formula in 64 bits (needs a B200).

Every slot of the pools that no sequence uses holds NaN, so reading one shows."""
import numpy as np
import pytest

import chunk_cases as cc
from helpers import dev

pytestmark = pytest.mark.gpu

SENTINEL = 77.0


EMPTY = 0


@pytest.fixture(params=[0, 150], ids=["", "wide"], autouse=True)
def empty_sequences(request):
    """Every test runs as it is, and with 150 sequences without tokens behind its own (short prompts are worked on in units of one
    slot where the GPU has an SM for each, else of two)."""
    global EMPTY
    EMPTY = request.param
    yield
    EMPTY = 0


def case(lens, hq, hkv, page, seed, pad=0, width=None):
    rng = np.random.default_rng(seed)
    k, v, table = cc.paged(lens, hkv, page, rng, width=width)
    q = rng.standard_normal((int(cc.starts(lens)[-1]) + pad, hq, cc.D)).astype(np.float16)
    return q, k, v, table


def call(i4, cuda, q, k, v, table, lens, **kw):
    import torch
    out = torch.full(q.shape, SENTINEL, dtype=torch.float16, device=cuda)
    lens = list(lens) + [(0, 0)] * EMPTY
    table = np.concatenate([table, np.full((EMPTY, table.shape[1]), -1, dtype=np.int32)])
    i4.paged_gqa_chunk(dev(q, cuda), dev(k, cuda), dev(v, cuda), dev(table, cuda), dev(cc.starts(lens), cuda),
                       dev(np.array([c for _, c in lens], dtype=np.int32), cuda), out=out, **kw)
    torch.cuda.synchronize()
    assert i4.device_error() == 0
    return out.cpu().numpy()


def check(got, q, k, v, table, lens, page, window=0, scale=None):
    n = int(cc.starts(lens)[-1])
    want, bound = cc.attention(q[:n], k, v, table, lens, page, window, scale)
    assert np.all(np.isfinite(got[:n])), np.argwhere(~np.isfinite(got[:n]))[:5]
    off = np.abs(got[:n].astype(np.float64) - want) - bound
    assert off.max(initial=-1.0) <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    assert np.all(got[n:] == SENTINEL)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 2)], [(1, 127)], [(1, 128)], [(1, 129)], [(1, 700)], [(2, 2)], [(17, 17)], [(18, 18)], [(19, 300)],
    [(37, 37)], [(130, 130)], [(129, 385)],
])
def test_one_sequence(i4lib, cuda, lens, page):
    q, k, v, table = case(lens, 7, 1, page, seed=page + lens[0][1])
    check(call(i4lib, cuda, q, k, v, table, lens), q, k, v, table, lens, page)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (6, 2), (4, 1), (5, 1), (12, 2), (28, 4), (16, 2), (8, 8)])
def test_head_layouts(i4lib, cuda, hq, hkv):
    lens = [(1, 300), (40, 41), (5, 260)]
    q, k, v, table = case(lens, hq, hkv, 16, seed=hq)
    check(call(i4lib, cuda, q, k, v, table, lens, max_q=40), q, k, v, table, lens, 16)


@pytest.mark.parametrize("max_q", [0, 1, 150])
def test_ragged_batch_with_empty_sequences_and_rows_behind(i4lib, cuda, max_q):
    lens = [(0, 50), (1, 513), (150, 150), (0, 0), (3, 3), (1, 1), (64, 900), (0, 7), (1, 1025), (33, 34), (0, 9)]
    q, k, v, table = case(lens, 14, 2, 32, seed=5, pad=9)
    check(call(i4lib, cuda, q, k, v, table, lens, max_q=max_q), q, k, v, table, lens, 32)


@pytest.mark.parametrize("n_seq", [33, 70, 1100])
def test_many_sequences(i4lib, cuda, n_seq):
    rng = np.random.default_rng(n_seq)
    lens = [(int(a), int(a + b)) for a, b in zip(rng.integers(0, 3, n_seq), rng.integers(0, 40, n_seq))]
    q, k, v, table = case(lens, 4, 2, 8, seed=n_seq, pad=2)
    check(call(i4lib, cuda, q, k, v, table, lens, max_q=2), q, k, v, table, lens, 8)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("hq,hkv,lens", [
    (7, 1, [(700, 4000), (40, 3000), (19, 6001), (37, 900), (1, 5000), (36, 2500)]),
    (40, 20, [(200, 200), (130, 700), (65, 70), (64, 64)]),
    (12, 12, [(300, 300), (129, 130), (128, 1000), (257, 400)]),
])
def test_units_of_two_slots(i4lib, cuda, hq, hkv, lens, window):
    """Too much for units of one slot: units whose second slot is full, has a token or has none."""
    q, k, v, table = case(lens, hq, hkv, 32, seed=hq + window, pad=3)
    check(call(i4lib, cuda, q, k, v, table, lens, window=window), q, k, v, table, lens, 32, window)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 300, 5000])
def test_window(i4lib, cuda, window):
    lens = [(1, 900), (260, 700), (20, 20), (1, 50)]
    q, k, v, table = case(lens, 4, 2, 16, seed=window)
    check(call(i4lib, cuda, q, k, v, table, lens, window=window), q, k, v, table, lens, 16, window)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 9])
def test_widest_window(i4lib, cuda, window):
    """Also where a chunk begins at negative positions: the window's first position stays a number of 32 bits."""
    lens = [(40, 10), (1, 300), (9, 9), (200, 150)]
    q, k, v, table = case([(40, 40), (1, 300), (9, 9), (200, 200)], 7, 1, 16, seed=12)
    check(call(i4lib, cuda, q, k, v, table, lens, window=window), q, k, v, table, lens, 16)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 65504.0])
def test_what_a_row_does_not_see_does_not_reach_it(i4lib, cuda, bad):
    """K and V of later tokens of the chunk, and of tokens before the window, hold NaN or infinity: the rows that do not
    see them stay right; the last row sees the last token's K and V and is left out."""
    lens, window = [(50, 400), (1, 300)], 64
    q, k, v, table = case(lens, 7, 1, 16, seed=3)
    clean = (k.copy(), v.copy())
    seq0 = lambda t: (table[0, t // 16], slice(None), t % 16)  # noqa: E731
    for t in list(range(0, 350 - window + 1)) + [399]:
        k[seq0(t)] = bad
        v[seq0(t)] = bad
    for t in range(0, 300 - window):
        v[table[1, t // 16], :, t % 16] = bad
    got = call(i4lib, cuda, q, k, v, table, lens, window=window)
    want, bound = cc.attention(q, *clean, table, lens, 16, window)
    rows = [i for i in range(51) if i != 49]
    # row i < 49 at position 350 + i sees 287 + i .. 350 + i: all clean
    assert np.all(np.abs(got[rows].astype(np.float64) - want[rows]) <= bound[rows])


def test_positions_that_do_not_exist_give_zeros(i4lib, cuda):
    """ctx_len below the number of rows: the first rows stand at negative positions and see nothing."""
    lens = [(6, 6), (9, 4), (3, 0)]
    q, k, v, table = case([(6, 6), (9, 9), (3, 3)], 7, 1, 8, seed=1)
    got = call(i4lib, cuda, q, k, v, table, lens)
    assert np.all(got[6:11] == 0) and np.all(got[15:18] == 0)
    check(got, q, k, v, table, lens, 8)


def test_positions_behind_the_table_row_are_not_seen(i4lib, cuda):
    q, k, v, table = case([(4, 32)], 7, 1, 16, seed=2)
    got = call(i4lib, cuda, q, k, v, table, [(4, 40)])  # positions 36..39, the row holds 32
    for i in range(4):
        want, bound = cc.attention(q[i:i + 1], k, v, table, [(1, 32)], 16)
        assert np.all(np.abs(got[i].astype(np.float64) - want[0]) <= bound[0])


@pytest.mark.parametrize("entry", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_page_id_outside_the_pools_reads_as_zeros(i4lib, cuda, entry):
    lens = [(3, 50)]
    q, k, v, table = case(lens, 4, 2, 16, seed=9)
    hole = table[0, 1]
    k2, v2 = k.copy(), v.copy()
    k2[hole], v2[hole] = 0, 0
    want, bound = cc.attention(q, k2, v2, table, lens, 16)
    bad = table.copy()
    bad[0, 1] = entry
    got = call(i4lib, cuda, q, k, v, bad, lens)
    assert np.all(np.abs(got.astype(np.float64) - want) <= bound)


def test_long_context_is_split_and_joined(i4lib, cuda):
    """Few rows over a long context: the work of one row is spread over the GPU."""
    lens = [(2, 20011)]
    q, k, v, table = case(lens, 7, 1, 64, seed=4)
    q[0] *= 4  # a sharper row: its maximum moves as the context goes on
    check(call(i4lib, cuda, q, k, v, table, lens, max_q=2), q, k, v, table, lens, 64)


def test_rising_scores(i4lib, cuda):
    """Scores that grow along the context, by more than 2^8 in the exponential from tile to tile, and then fall."""
    lens = [(20, 1200)]
    q, k, v, table = case(lens, 4, 1, 16, seed=6)
    q[:] = np.abs(q)
    ramp = np.concatenate([np.linspace(-4, 4, 900), np.linspace(4, -4, 300)])
    for t in range(1200):
        k[table[0, t // 16], :, t % 16] = np.float16(ramp[t])
    check(call(i4lib, cuda, q, k, v, table, lens), q, k, v, table, lens, 16)


@pytest.mark.parametrize("scale", [1e-3, 0.5, 2.0])
def test_scale(i4lib, cuda, scale):
    lens = [(9, 200)]
    q, k, v, table = case(lens, 4, 1, 16, seed=8)
    check(call(i4lib, cuda, q, k, v, table, lens, scale=scale), q, k, v, table, lens, 16, scale=scale)


def test_strided_rows(i4lib, cuda):
    import torch
    lens = [(5, 90), (30, 30)]
    q, k, v, table = case(lens, 6, 2, 16, seed=7)
    wide = torch.full((35, 6 * 128 + 40), float("nan"), dtype=torch.float16, device=cuda)
    wide[:, 8:8 + 768] = dev(q, cuda).view(35, -1)
    view = wide[:, 8:8 + 768].view(35, 6, 128)
    args = [dev(a, cuda) for a in (k, v, table, cc.starts(lens), np.array([90, 30], dtype=np.int32))]
    got = i4lib.paged_gqa_chunk(view, *args)
    same = i4lib.paged_gqa_chunk(dev(q, cuda), *args)
    assert torch.equal(got, same)
    check(got.cpu().numpy(), q, k, v, table, lens, 16)


def test_same_bits_every_time_and_with_any_workspace(i4lib, cuda):
    import torch
    lens = [(1, 3000), (200, 777), (1, 12)]
    q, k, v, table = case(lens, 14, 2, 16, seed=12)
    a = call(i4lib, cuda, q, k, v, table, lens)
    for fill in (0, 255):
        ws = torch.full((i4lib.paged_gqa_chunk_ws_bytes(),), fill, dtype=torch.uint8, device=cuda)
        for _ in range(3):
            assert np.array_equal(call(i4lib, cuda, q, k, v, table, lens, ws=ws).view(np.uint16), a.view(np.uint16))


def test_any_page_order_gives_the_same_bits(i4lib, cuda):
    lens = [(40, 500)]
    q, k, v, table = case(lens, 7, 1, 16, seed=13)
    a = call(i4lib, cuda, q, k, v, table, lens)
    perm = np.random.default_rng(0).permutation(k.shape[0])
    k2, v2 = np.empty_like(k), np.empty_like(v)
    k2[perm], v2[perm] = k, v
    table2 = np.where(table >= 0, perm[table], -1).astype(np.int32)
    assert np.array_equal(call(i4lib, cuda, q, k2, v2, table2, lens).view(np.uint16), a.view(np.uint16))


def test_captured_call_follows_the_lengths(i4lib, cuda):
    """One captured call, replayed as the lengths and the cut into sequences change."""
    import torch
    q, k, v, table = case([(20, 600), (30, 300)], 7, 1, 16, seed=14)
    tq, tk, tv, tt = (dev(a, cuda) for a in (q, k, v, table))
    start = torch.tensor([0, 20, 50], dtype=torch.int32, device=cuda)
    ctx = torch.tensor([600, 300], dtype=torch.int32, device=cuda)
    ws = torch.empty(i4lib.paged_gqa_chunk_ws_bytes(), dtype=torch.uint8, device=cuda)
    out = torch.full((50, 7, 128), SENTINEL, dtype=torch.float16, device=cuda)
    run = lambda: i4lib.paged_gqa_chunk(tq, tk, tv, tt, start, ctx, out=out, ws=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for lens in ([(20, 600), (30, 300)], [(1, 350), (2, 2)], [(0, 0), (50, 100)], [(44, 44), (0, 300)]):
        start.copy_(torch.from_numpy(cc.starts(lens)))
        ctx.copy_(torch.tensor([c for _, c in lens], dtype=torch.int32))
        out.fill_(SENTINEL)
        g.replay()
        torch.cuda.synchronize()
        check(out.cpu().numpy(), q, k, v, table, lens, 16)


@pytest.mark.parametrize("starts", [[0, 500, 0, 500], [0, 500] * 20, [500, 0] * 450, [0, 300, 200] + [500] * 30,
                                    [-5, 100, 2 ** 31 - 1, -2 ** 31, 400]])
def test_starts_that_decrease_stay_within_the_rows(i4lib, cuda, starts):
    """Sequences that claim the same rows, or rows that do not exist: whatever comes of it, nothing is written behind the rows and
    the next call is right."""
    import torch
    T, n_seq = 500, len(starts) - 1
    lens = [(T, 600)]
    q, k, v, table = case(lens, 7, 1, 16, seed=31)
    buf = torch.full((T + 64, *q.shape[1:]), SENTINEL, dtype=torch.float16, device=cuda)
    ctx = torch.full((n_seq,), 600, dtype=torch.int32, device=cuda)
    i4lib.paged_gqa_chunk(dev(q, cuda), dev(k, cuda), dev(v, cuda), dev(np.tile(table, (n_seq, 1)), cuda),
                          dev(np.array(starts, dtype=np.int32), cuda), ctx, out=buf[:T])
    torch.cuda.synchronize()
    assert i4lib.device_error() == 0
    assert (buf[T:] == SENTINEL).all()
    check(call(i4lib, cuda, q, k, v, table, lens), q, k, v, table, lens, 16)


def test_two_streams_with_their_own_workspaces(i4lib, cuda):
    import torch
    sets = []
    for seed in (20, 21):
        lens = [(1, 2000 + seed), (60, 100)]
        q, k, v, table = case(lens, 7, 1, 16, seed=seed)
        args = [dev(a, cuda) for a in (q, k, v, table, cc.starts(lens), np.array([c for _, c in lens], dtype=np.int32))]
        ws = torch.empty(i4lib.paged_gqa_chunk_ws_bytes(), dtype=torch.uint8, device=cuda)
        sets.append((lens, (q, k, v, table), args, ws, torch.cuda.Stream(), torch.empty_like(args[0])))
    torch.cuda.synchronize()
    for _ in range(20):
        for _, _, args, ws, stream, out in sets:
            i4lib.paged_gqa_chunk(*args, out=out, ws=ws, stream=stream)
    torch.cuda.synchronize()
    for lens, host, _, _, _, out in sets:
        check(out.cpu().numpy(), *host, lens, 16)


def test_same_as_the_decode_kernel(i4lib, cuda):
    """Single tokens: the values of paged_gqa_decode, each within its own bound."""
    import torch
    lens = [(1, c) for c in (1, 17, 512, 3001)]
    q, k, v, table = case(lens, 28, 4, 16, seed=30)
    got = call(i4lib, cuda, q, k, v, table, lens, max_q=1)
    ctx = dev(np.array([c for _, c in lens], dtype=np.int32), cuda)
    clean = [torch.nan_to_num(dev(a, cuda)) for a in (k, v)]
    ref = i4lib.paged_gqa_decode(dev(q, cuda), *clean, dev(np.maximum(table, 0), cuda), ctx).cpu().numpy()
    _, bound = cc.attention(q, k, v, table, lens, 16)
    assert np.all(np.abs(got.astype(np.float64) - ref) <= 2 * bound)


def test_calls_that_allocate_on_another_stream(i4lib, cuda):
    """Output and workspace made by the call, on a stream that is not the current one, while the current one keeps
    allocating and overwriting what is given back."""
    import torch
    lens = [(1, 4000), (90, 90)]
    q, k, v, table = case(lens, 7, 1, 16, seed=40)
    args = [dev(a, cuda) for a in (q, k, v, table, cc.starts(lens), np.array([c for _, c in lens], dtype=np.int32))]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(20):
        outs.append(i4lib.paged_gqa_chunk(*args, stream=side))
        for _ in range(3):
            torch.full((i4lib.paged_gqa_chunk_ws_bytes() // 4,), float("nan"), device=cuda)
    torch.cuda.synchronize()
    for out in outs:
        check(out.cpu().numpy(), q, k, v, table, lens, 16)


def gpu_reference(q, k, v, scale=None):
    """64-bit attention of rows q [Hq][128] over k, v [ctx][128] on the GPU, and the bound of cc.attention."""
    import torch
    scale = 1 / np.sqrt(cc.D) if scale is None else scale
    qd, kd, vd = q.double(), k.double(), v.double()
    p = torch.softmax(qd @ kd.T * scale, dim=1)
    out, a = p @ vd, p @ vd.abs()
    e = 128 * 2.0 ** -23 * scale * (qd.abs() @ kd.abs().T).amax(dim=1, keepdim=True)
    bound = 2.0 ** -11 * (a + out.abs()) + 2 * e * a + 2.0 ** -13 * a + 2.0 ** -25 * (vd.abs().sum(0) + 1)
    return out, bound


def test_a_million_positions(i4lib, cuda):
    """The longest row of the page table. A row's sums pass 8192 tiles instead of the 2^9 additions of cc.attention's
    bound: 2^-23 * 8192 * A = 2^-10 A more."""
    import torch
    ctx, page = 1 << 20, 128
    gen = torch.Generator(device=cuda).manual_seed(1)
    k, v = (torch.randn((ctx // page, 1, page, 128), generator=gen, device=cuda, dtype=torch.float16) for _ in range(2))
    q = torch.randn((2, 4, 128), generator=gen, device=cuda, dtype=torch.float16)
    perm = torch.randperm(ctx // page, generator=gen, device=cuda)
    table = perm.to(torch.int32)[None].contiguous()
    start, n = torch.tensor([0, 2], dtype=torch.int32, device=cuda), torch.tensor([ctx], dtype=torch.int32, device=cuda)
    got = i4lib.paged_gqa_chunk(q, k, v, table, start, n, max_q=2)
    kk, vv = (t[perm][:, 0].reshape(-1, 128) for t in (k, v))
    for i in range(2):
        want, bound = gpu_reference(q[i], kk[:ctx - 1 + i], vv[:ctx - 1 + i])
        a = (bound / 2.0 ** -11).abs()  # at least A
        assert bool(((got[i].double() - want).abs() <= bound + 2.0 ** -10 * a).all())
    assert i4lib.device_error() == 0


def test_pools_behind_32_bits(i4lib, cuda):
    """Pages whose values lie more than 2^32 bytes and 2^31 values into the pools: attention, append and copy."""
    import torch
    pages, page = (1 << 31) // (2 * 128 * 128) + 70, 128
    f16, i32 = torch.float16, torch.int32
    k, v = (torch.empty((pages, 2, page, 128), dtype=f16, device=cuda) for _ in range(2))
    assert k.numel() > 1 << 31
    gen = torch.Generator(device=cuda).manual_seed(2)
    ids = [pages - 1, 3, pages - 60, pages - 2]
    for t in (k, v):
        t[ids] = torch.randn((4, 2, page, 128), generator=gen, device=cuda, dtype=f16)
    q = torch.randn((3, 4, 128), generator=gen, device=cuda, dtype=f16)
    table = torch.tensor([ids], dtype=i32, device=cuda)
    start, n = torch.tensor([0, 3], dtype=i32, device=cuda), torch.tensor([500], dtype=i32, device=cuda)
    cs = i4lib.rope_table(512, 128)
    qkv = torch.randn((3, 8 * 128), generator=gen, device=cuda, dtype=f16)
    i4lib.rope_append_chunk(qkv, start, n, cs, 4, 2, k, v, table)
    assert torch.equal(v[pages - 2, :, 113:116].transpose(0, 1).reshape(3, -1), qkv[:, 6 * 128:])
    got = i4lib.paged_gqa_chunk(q, k, v, table, start, n)
    for i in range(3):
        for h in range(4):
            kk, vv = (t[ids, h // 2].reshape(-1, 128)[:498 + i] for t in (k, v))
            want, bound = gpu_reference(q[i, h:h + 1], kk, vv)
            assert bool(((got[i, h].double() - want[0]).abs() <= bound[0]).all())
    i4lib.kv_pages_copy([k, v], table[0, :1].contiguous(), torch.tensor([pages - 70], dtype=i32, device=cuda))
    assert torch.equal(k[pages - 70], k[pages - 1]) and torch.equal(v[pages - 70], v[pages - 1])
