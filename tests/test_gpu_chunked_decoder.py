"""Chunks of prompts, forks, single tokens, freed and compacted pages in one run of a small decoder, against the oracle
(needs a B200)."""
import numpy as np
import pytest

import oracle
from int4_weight_only_02_b200 import synth
from helpers import normwise_err

pytestmark = pytest.mark.gpu

SHAPE = synth.ModelShape(layers=2, hidden=512, inter=1024, n_q=4, n_kv=2, head_dim=128, vocab=2048, group=128, page_size=16,
                         max_ctx=256)


@pytest.fixture(scope="module")
def parts():
    return [synth.layer_weights(SHAPE, i, 4) for i in range(SHAPE.layers)], synth.global_weights(SHAPE, 4)


@pytest.fixture(scope="module")
def model(i4lib, cuda, parts):
    return i4lib.DeviceModel(SHAPE, *parts, device=cuda)


def oracle_logits(parts, tokens):
    dec = oracle.DecoderOracle(SHAPE, *parts, synth.page_table(SHAPE, 5), num_pages=SHAPE.max_pages)
    return dec.forward(np.asarray(tokens), 0)[0]


class Text:
    """What a sequence was fed, beside what the decoder says of it: its logits after any chunk are the oracle's after all its
    tokens at once."""

    def __init__(self, parts):
        self.parts, self.tokens = parts, {}

    def check(self, seqs, nxt, logits):
        for k, t, row in zip(sorted(seqs), nxt.cpu().tolist(), logits.cpu().numpy()):
            want = oracle_logits(self.parts, self.tokens[k])
            # fp16 stores all along two layers: the bound that the prefill's logits are held to
            assert normwise_err(row, want) <= 1e-2, k
            assert t == int(np.argmax(row))

    def feed(self, dec, chunks):
        for k, v in chunks.items():
            self.tokens[k] = list(self.tokens.get(k, [])) + list(map(int, v))
        nxt, logits = dec.run(chunks)
        self.check(chunks, nxt, logits)
        return dict(zip(sorted(chunks), nxt.cpu().tolist()))


def test_a_serving_run(i4lib, cuda, parts, model):
    cache = i4lib.PagedCache(model, n_seqs=6, num_pages=40)
    dec = i4lib.ChunkedDecoder(model, cache, max_tokens=128)
    text = Text(parts)
    prompt = [synth.prompt_tokens(SHAPE, n, seed=10 + i) for i, n in enumerate((70, 23, 41))]
    text.feed(dec, {0: prompt[0][:37], 3: prompt[1]})                    # two prompts, one of them in chunks
    nxt = text.feed(dec, {0: prompt[0][37:], 3: [5], 1: prompt[2][:1]})  # the rest beside single tokens
    nxt = text.feed(dec, {0: [nxt[0]], 3: [nxt[3]], 1: prompt[2][1:]})
    # two continuations of sequence 0 that go on with other tokens than it does
    assert cache.fork([0, 0], [4, 2]).cpu().tolist() == [0, 0]
    text.tokens[4], text.tokens[2] = list(text.tokens[0]), list(text.tokens[0])
    nxt = text.feed(dec, {0: [nxt[0]], 2: [11], 4: [12, 13, 14], 1: [nxt[1]]})
    cache.free([3])
    text.tokens[3] = []
    n_live = int(cache.compact().item())
    held = [-(-len(text.tokens[k]) // 16) for k in (0, 1, 2, 4)]
    assert n_live == sum(held) - 2 * 4  # sequences 0, 2 and 4 share the four pages of the first 64 tokens
    assert torch_refs(cache)[:n_live].min() == 1 and torch_refs(cache)[n_live:].max() == 0
    for _ in range(3):
        nxt = text.feed(dec, {k: [nxt[k]] for k in (0, 1, 2, 4)})
    nxt.update(text.feed(dec, {3: prompt[1][:9], 5: prompt[0][:50]}))    # a freed slot and a new one
    text.feed(dec, {k: [nxt[k]] for k in range(6)})
    assert i4lib.device_error() == 0


def torch_refs(cache):
    return cache.refs.cpu().numpy()


def test_no_pages_leaves_the_cache_as_it_was(i4lib, cuda, parts, model):
    cache = i4lib.PagedCache(model, n_seqs=3, num_pages=5)
    dec = i4lib.ChunkedDecoder(model, cache, max_tokens=128)
    text = Text(parts)
    prompt = synth.prompt_tokens(SHAPE, 90, seed=3)
    nxt = text.feed(dec, {0: prompt[:30], 1: prompt[:17]})
    state = [t.clone() for t in (cache.page_table, cache.ctx_len, cache.refs)]
    with pytest.raises(i4lib.I4Error, match="no pages"):
        dec.run({0: prompt[30:40], 1: [3], 2: prompt[:40]})
    for a, b in zip(state, (cache.page_table, cache.ctx_len, cache.refs)):
        assert np.array_equal(a.cpu().numpy(), b.cpu().numpy())
    nxt = text.feed(dec, {0: [nxt[0]], 1: [nxt[1]]})
    cache.free([1])
    text.feed(dec, {0: [nxt[0]], 2: prompt[:40]})


def test_cache_calls_on_a_stream_that_is_behind(i4lib, cuda, model):
    """The lists that a call makes of its arguments live until its stream has read them."""
    import torch
    cache = i4lib.PagedCache(model, n_seqs=6, num_pages=40)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    status = [cache.reserve([3, 1, 0], [20, 16, 33], stream=side), cache.fork([3, 1], [2, 4], stream=side)]
    cache.free([1], stream=side)
    over = [torch.full((k,), -7, dtype=torch.int32, device=cuda) for k in (1, 2, 3) for _ in range(8)]
    torch.cuda.synchronize()
    assert [s.cpu().tolist() for s in status] == [[0, 0, 0], [0, 0]] and len(over) == 24
    assert cache.ctx_len.cpu().tolist() == [33, 0, 20, 20, 16, 0]
    assert [len(row[row >= 0]) for row in cache.page_table.cpu()] == [3, 0, 2, 2, 1, 0]


def test_refusals(i4lib, cuda, model):
    cache = i4lib.PagedCache(model, n_seqs=2, num_pages=20)
    dec = i4lib.ChunkedDecoder(model, cache, max_tokens=16)
    for chunks in ({}, {2: [1]}, {-1: [1]}, {0: []}, {0: list(range(9)), 1: list(range(8))}):
        with pytest.raises(ValueError):
            dec.run(chunks)
    assert int(cache.ctx_len.sum().item()) == 0


def test_extended_context(i4lib, cuda, parts, model):
    """Scaled positions change the logits and stay the same whether the prompt comes whole or in chunks."""
    prompt = synth.prompt_tokens(SHAPE, 60, seed=8)
    got = []
    for cuts in ([60], [13, 31, 60]):
        cache = i4lib.PagedCache(model, n_seqs=1, num_pages=8)
        dec = i4lib.ChunkedDecoder(model, cache, max_tokens=64, scaling="yarn", factor=4.0, original_ctx=64)
        at = 0
        for c in cuts:
            _, logits = dec.run({0: prompt[at:c]})
            at = c
        got.append(logits[0].cpu().numpy())
    assert normwise_err(got[1], got[0]) <= 1e-2
    assert normwise_err(got[0], oracle_logits(parts, prompt)) > 1e-2


def state_of(cache):
    return [t.cpu().numpy() for t in (cache.page_table, cache.ctx_len, cache.refs)]


def same_state(cache, state):
    for a, b in zip(state, state_of(cache)):
        assert np.array_equal(a, b)


def test_more_tokens_than_the_row_holds(i4lib, cuda, parts, model):
    """Not a lack of pages: freeing some would not help, so it is another error; what was granted is given back."""
    cache = i4lib.PagedCache(model, n_seqs=3, num_pages=30, max_pages_per_seq=3)
    dec = i4lib.ChunkedDecoder(model, cache, max_tokens=64)
    text = Text(parts)
    prompt = synth.prompt_tokens(SHAPE, 60, seed=4)
    nxt = text.feed(dec, {0: prompt[:47], 1: prompt[:5]})
    text.feed(dec, {0: [nxt[0]]})  # the row is full
    state = state_of(cache)
    for chunks in ({0: [1]}, {0: [1], 1: prompt[:20], 2: [3]}, {2: prompt[:49]}):
        with pytest.raises(i4lib.I4Error, match="48 positions") as e:
            dec.run(chunks)
        assert e.value.status == i4lib.I4_EINVAL
        same_state(cache, state)
    text.feed(dec, {1: [nxt[1]], 2: prompt[:48]})


@pytest.mark.parametrize("at", ["embed_gather", "rope_append_chunk", "silu_mul", "argmax_rows"])
def test_a_call_that_fails_leaves_the_cache_as_it_was(i4lib, cuda, parts, model, monkeypatch, at):
    cache = i4lib.PagedCache(model, n_seqs=3, num_pages=30)
    dec = i4lib.ChunkedDecoder(model, cache, max_tokens=64)
    text = Text(parts)
    prompt = synth.prompt_tokens(SHAPE, 60, seed=5)
    nxt = text.feed(dec, {0: prompt[:30], 2: prompt[:17]})
    state = state_of(cache)

    def fails(*a, **kw):
        raise i4lib.I4Error(i4lib.I4_EINVAL, "made to fail")

    with monkeypatch.context() as m:
        m.setattr(i4lib, at, fails)
        with pytest.raises(i4lib.I4Error, match="made to fail"):
            dec.run({0: [nxt[0]], 1: prompt[:33], 2: [1, 2, 3]})
    same_state(cache, state)
    nxt = text.feed(dec, {0: [nxt[0]], 1: prompt[:33], 2: [nxt[2]]})
    text.feed(dec, {k: [nxt[k]] for k in range(3)})


def test_a_cache_of_another_model_is_refused(i4lib, cuda, model, parts):
    import dataclasses
    for change in (dict(page_size=8), dict(layers=1), dict(n_kv=4)):
        other = dataclasses.replace(SHAPE, **change)
        weights = [synth.layer_weights(other, i, 4) for i in range(other.layers)], synth.global_weights(other, 4)
        cache = i4lib.PagedCache(i4lib.DeviceModel(other, *weights, device=cuda), n_seqs=2, num_pages=8)
        with pytest.raises(ValueError, match="cache"):
            i4lib.ChunkedDecoder(model, cache, max_tokens=16)


@pytest.mark.parametrize("device", ["cuda", "cuda:0"])
def test_a_model_whose_device_is_a_name(i4lib, cuda, parts, device):
    model = i4lib.DeviceModel(SHAPE, *parts, device=device)
    dec = i4lib.ChunkedDecoder(model, i4lib.PagedCache(model, n_seqs=2, num_pages=8), max_tokens=16)
    text = Text(parts)
    nxt = text.feed(dec, {1: [3, 1, 4]})
    text.feed(dec, {0: [1, 5], 1: [nxt[1]]})
