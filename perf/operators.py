"""Measured cases of the chunked serving operators over a paged fp16 cache.

Kinds of case:

* ``attn``     attention of a ragged batch of new tokens over pages (``paged_gqa_chunk``);
* ``rope``     rotary positions of a ragged batch and the append of its K/V (``rope_append_chunk``);
* ``fork``     sequences that continue others: shared pages and a copied last page (``kv_pages_fork``);
* ``compact``  moving the pages in use to the front of the pools (``kv_pages_compact``).

``run`` computes each in elementary torch operations, or, with ``own``, by the framework's calls.
"""
import math
import random

import torch

own = False

D = 128
MOST_PAIRS = 8192 * 8193 // 2 * 28  # (query head, position) pairs of the largest prompt
MOST_KEPT = 1 << 20  # (kv head, position) pairs kept in the pages of a drawn case


def listed():
    return [
        # a decode step of a small batch: one token a sequence, latency counts
        dict(name="attn 4 single tokens", kind="attn", lens="1:514,1:77,1:1000,1:2049", hq=28, hkv=4, page=16, window=0, pad=0),
        # the prompt of the benchmark's time to first token
        dict(name="attn prompt 512", kind="attn", lens="512:512", hq=28, hkv=4, page=16, window=0, pad=0),
        # one chunk of a long prompt whose beginning is cached already
        dict(name="attn 512 behind 32k", kind="attn", lens="512:32768", hq=28, hkv=4, page=64, window=0, pad=0),
        # mixed step of a server: single tokens beside odd chunks, a sliding window, rows behind the last sequence
        dict(name="attn mixed window", kind="attn", lens="1:4093,301:2348,1:17,1:8191,777:777,64:5000,0:100,1:1,130:1111,1:6000",
             hq=32, hkv=4, page=32, window=2000, pad=7),
        # a long prompt at once: dense work
        dict(name="attn prompt 8192", kind="attn", lens="8192:8192", hq=28, hkv=4, page=128, window=0, pad=0),
        # a decode step's rotation and append
        dict(name="rope 8 single tokens", kind="rope", lens="1:514,1:77,1:1000,1:2049,1:16,1:4000,1:1,1:333", hq=28, hkv=4, page=16,
             rd=128, inter=False, scaling="none", pad=0),
        # the benchmark's prompt, with the frequencies of a context extended four times
        dict(name="rope prompt 512 extended", kind="rope", lens="512:40000", hq=28, hkv=4, page=16, rd=128, inter=False, scaling="yarn",
             pad=0),
        # long chunks of several sequences, half the head rotated in interleaved pairs
        dict(name="rope 16k interleaved half", kind="rope", lens="8000:8000,5000:9001,3001:20000,383:383", hq=28, hkv=4, page=64, rd=64,
             inter=True, scaling="linear", pad=13),
        # a few alternatives of one sequence in a small decoder
        dict(name="fork 3 of 4 pools", kind="fork", pools=4, hkv=4, page=16, pages=256, seqs=8, ctx=203, forks=3),
        # 63 samples of one prompt, every layer of the 7B shape
        dict(name="fork 63 of 56 pools", kind="fork", pools=56, hkv=4, page=16, pages=768, seqs=64, ctx=4000 + 15, forks=63),
        # a small cache after a few sequences ended
        dict(name="compact 9 pages", kind="compact", pools=4, hkv=4, page=16, pages=64, live=40, moves=9, seqs=8),
        # a full cache of the 7B shape after half of it was freed
        dict(name="compact 300 pages", kind="compact", pools=56, hkv=4, page=16, pages=1500, live=700, moves=300, seqs=33),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "rope", "rope", "fork", "compact"])
    hq, hkv = rng.choice([(28, 4), (32, 4), (16, 16), (8, 4), (4, 1), (5, 1), (12, 2)])
    page = rng.choice([8, 16, 32, 64, 128])
    if kind == "attn":
        most, lens, pairs, kept = rng.choice([1, 64, 8192]), [], 0, 0
        for _ in range(_log(rng, 1, 24)):
            n = 1 if rng.random() < 0.2 else _log(rng, 1, most)
            ctx = n if rng.random() < 0.3 else n + _log(rng, 1, 32768 - n)
            if pairs + n * ctx * hq <= MOST_PAIRS and kept + ctx * hkv <= MOST_KEPT:
                pairs, kept = pairs + n * ctx * hq, kept + ctx * hkv
                lens.append("%d:%d" % (n, ctx))
        window = _log(rng, 1, 8192) if rng.random() < 0.3 else 0
        return dict(kind=kind, lens=",".join(lens or ["1:100"]), hq=hq, hkv=hkv, page=page, window=window, pad=rng.choice([0, 0, 5]))
    if kind == "rope":
        most, lens, tokens, kept = rng.choice([1, 600, 12000]), [], 0, 0
        for _ in range(_log(rng, 1, 24)):
            n = _log(rng, 1, most)
            ctx = n if rng.random() < 0.3 else n + _log(rng, 1, 50000 - n)
            if tokens + n <= 16384 and kept + ctx * hkv <= MOST_KEPT:
                tokens, kept = tokens + n, kept + ctx * hkv
                lens.append("%d:%d" % (n, ctx))
        return dict(kind=kind, lens=",".join(lens or ["1:100"]), hq=hq, hkv=hkv, page=page, rd=rng.choice([32, 64, 96, 128]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "yarn"]), pad=rng.choice([0, 0, 5]))
    pools, hkv, page = rng.choice([2, 4, 24, 56]), rng.choice([1, 2, 4]), rng.choice([8, 16, 32])
    if kind == "fork":
        forks, ctx = _log(rng, 1, 63), _log(rng, 2, 4000)
        seqs = forks + rng.randint(1, 9)
        return dict(kind=kind, pools=pools, hkv=hkv, page=page, pages=-(-ctx // page) + seqs * 3 + rng.randint(0, 99), seqs=seqs, ctx=ctx, forks=forks)
    pages = _log(rng, 24, 1500)
    live = rng.randint(pages // 4, pages // 2)
    return dict(kind=kind, pools=pools, hkv=hkv, page=page, pages=pages, live=live, moves=rng.randint(1, min(live, pages - live)),
                seqs=rng.randint(1, 40))


def _lens(case):
    return [tuple(int(v) for v in part.split(":")) for part in case["lens"].split(",")]


def _seen(n, ctx, window):
    """(position pairs, first position seen) of a chunk of n tokens that ends at ctx."""
    first = ctx - n
    if not window:
        return n * first + n * (n + 1) // 2, 0
    short = max(0, min(n, window - 1 - first))  # tokens that see fewer than `window` positions
    return short * first + short * (short + 1) // 2 + (n - short) * window, max(0, first - window + 1)


def work(case):
    kind = case["kind"]
    if kind in ("attn", "rope"):
        lens = _lens(case)
        tokens, hq, hkv = sum(n for n, _ in lens), case["hq"], case["hkv"]
        meta = 4 * (2 * len(lens) + 1)
    if kind == "attn":
        pairs = kv = 0
        for n, ctx in lens:
            p, lo = _seen(n, ctx, case["window"])
            if n:
                pairs, kv = pairs + p, kv + ctx - lo
        return {"bytes": 2 * tokens * hq * D * 2 + kv * hkv * D * 2 * 2 + 4 * kv // case["page"] + meta, "flops": 4 * D * hq * pairs}
    if kind == "rope":
        rows = tokens * (hq + 2 * hkv) * D * 2
        return {"bytes": 2 * rows + tokens * case["rd"] // 2 * 8 + meta, "flops": 3 * tokens * (hq + hkv) * case["rd"]}
    row = case["hkv"] * D * 2  # one token's K or V in one pool
    if kind == "fork":
        ctx, page = case["ctx"], case["page"]
        held = -(-ctx // page)
        return {"bytes": case["forks"] * (2 * case["pools"] * (ctx % page) * row + 4 * held) + 8 * held, "flops": 0}
    return {"bytes": 2 * case["moves"] * case["pools"] * case["page"] * row + 8 * case["live"] + 4 * case["pages"], "flops": 0}


def _tables(lens, page, gen, dev):
    """Pages of the sequences, in random order in one pool: (page table, pages of the pool)."""
    need = [-(-ctx // page) for _, ctx in lens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), max(max(need), 1)), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, pages


def _scaling(case):
    """(name, factor, positions of the original context) of a rotary case."""
    return {"none": ("none", 1.0, 0), "linear": ("linear", 4.0, 0), "yarn": ("yarn", 4.0, 32768)}[case["scaling"]]


def _frequencies(rd, theta, scaling, factor, original):
    """Angles a position, and the factor on cos and sin, in Python's 64 bits."""
    f = [theta ** (-2.0 * i / rd) for i in range(rd // 2)]
    if scaling == "linear":
        return [v / factor for v in f], 1.0
    if scaling == "yarn":
        def dim(turns):  # the pair that turns `turns` times over the original context
            return rd * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32)), 0), min(math.ceil(dim(1)), rd - 1)
        hi = hi + 0.001 if hi == lo else hi
        ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rd // 2)]
        return [v / factor * r + v * (1 - r) for v, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    return f, 1.0


THETA = 1.0e6
TABLE = 65536  # positions of the table of angles, made once like weights


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    kind, page, hkv = case["kind"], case["page"], case["hkv"]
    half = dict(dtype=torch.float16, device=dev)

    def normal(*shape):
        return torch.randn(shape, generator=gen, **half)

    if kind in ("attn", "rope"):
        lens, hq = _lens(case), case["hq"]
        tokens = sum(n for n, _ in lens)
        table, pages = _tables(lens, page, gen, dev)
        at = [0]
        for n, _ in lens:
            at.append(at[-1] + n)
        st = dict(case=case, lens=lens, at=at, table=table, q_start=torch.tensor(at, dtype=torch.int32, device=dev),
                  ctx_len=torch.tensor([c for _, c in lens], dtype=torch.int32, device=dev), max_q=max(n for n, _ in lens))
    if kind == "attn":
        st.update(q=normal(tokens + case["pad"], hq, D), k=normal(pages, hkv, page, D), v=normal(pages, hkv, page, D),
                  out=torch.zeros((tokens + case["pad"], hq, D), **half), ws=torch.zeros(64 << 20, dtype=torch.uint8, device=dev))
        return st
    if kind == "rope":
        scaling, factor, original = _scaling(case)
        f, m = _frequencies(case["rd"], THETA, scaling, factor, original)
        angle = torch.arange(TABLE, dtype=torch.float64, device=dev)[:, None] * torch.tensor(f, dtype=torch.float64, device=dev)
        st.update(qkv=normal(tokens + case["pad"], (hq + 2 * hkv) * D), k=normal(pages, hkv, page, D), v=normal(pages, hkv, page, D),
                  q_out=torch.zeros((tokens + case["pad"], hq, D), **half),
                  cs=torch.stack([angle.cos() * m, angle.sin() * m], dim=2).to(torch.float32))
        return st

    # a cache of several sequences; every pool of every layer has the same pages
    kv = normal(case["pools"], case["pages"], hkv, page, D)
    rng = random.Random(seed)
    seqs = case["seqs"]
    if kind == "fork":
        ctx, forks = case["ctx"], case["forks"]
        held = -(-ctx // page)
        ids = list(range(case["pages"]))
        rng.shuffle(ids)
        rows, refs, lens = [[-1] * (held + 1) for _ in range(seqs)], [0] * case["pages"], [0] * seqs
        order = list(range(seqs))
        rng.shuffle(order)
        src, dst = order[0], order[1:1 + forks]
        rows[src][:held], lens[src] = ids[:held], ctx
        for s in dst[::2]:  # every other one holds a page of an earlier text, which the fork gives back
            rows[s][0], lens[s] = ids[held + s], min(3, page)
        for s in range(seqs):
            for p in rows[s]:
                if p >= 0:
                    refs[p] += 1
        st = dict(src=torch.tensor([src] * forks, dtype=torch.int32, device=dev), dst=torch.tensor(dst, dtype=torch.int32, device=dev),
                  status=torch.zeros(forks, dtype=torch.int32, device=dev))
    else:
        live, moves = case["live"], case["moves"]
        ids = rng.sample(range(live), live - moves) + rng.sample(range(live, case["pages"]), moves)
        rng.shuffle(ids)
        cut = sorted(rng.randint(0, live) for _ in range(seqs - 1))
        parts = [ids[a:b] for a, b in zip([0] + cut, cut + [live])]
        width = live + 2
        rows, refs, lens = [p + [-1] * (width - len(p)) for p in parts], [0] * case["pages"], []
        for p in parts:
            lens.append(max(0, len(p) * page - rng.randrange(page)))
        for p in ids:
            refs[p] = 1
        st = dict(n_live=torch.zeros(1, dtype=torch.int32, device=dev))
    i32 = dict(dtype=torch.int32, device=dev)
    st.update(case=case, kv=kv, pools=list(kv), table=torch.tensor(rows, **i32), refs=torch.tensor(refs, **i32), ctx_len=torch.tensor(lens, **i32),
              ws=torch.zeros(1 << 20, dtype=torch.uint8, device=dev))
    st.update(table0=st["table"].clone(), refs0=st["refs"].clone())
    return st


# ------------------------------------------------------------------ plain forms

def _plain_attn(st):
    case, page = st["case"], st["case"]["page"]
    hkv, window, out = case["hkv"], case["window"], st["out"]
    group = case["hq"] // hkv
    dev = out.device
    for b, (n, ctx) in enumerate(st["lens"]):
        if n == 0:
            continue
        ids = st["table"][b, :-(-ctx // page)].long()
        k = st["k"][ids].permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :ctx].float()
        v = st["v"][ids].permute(1, 0, 2, 3).reshape(hkv, -1, D)[:, :ctx].float()
        q = st["q"][st["at"][b]:st["at"][b] + n].float().view(n, hkv, group, D).permute(1, 2, 0, 3)
        s = torch.matmul(q, k[:, None].transpose(2, 3)) * (1.0 / math.sqrt(D))
        pos, t = torch.arange(ctx - n, ctx, device=dev)[:, None], torch.arange(ctx, device=dev)
        hidden = t > pos
        if window:
            hidden = hidden | (t <= pos - window)
        s.masked_fill_(hidden, -math.inf)
        p = torch.exp(s - s.amax(dim=-1, keepdim=True))
        o = torch.matmul(p, v[:, None]) / p.sum(dim=-1, keepdim=True)
        out[st["at"][b]:st["at"][b] + n] = o.permute(2, 0, 1, 3).reshape(n, -1, D).half()
    return out


def _plain_rope(st):
    case, page = st["case"], st["case"]["page"]
    hq, hkv, rd = case["hq"], case["hkv"], case["rd"]
    tokens, dev = st["at"][-1], st["qkv"].device
    row = torch.arange(tokens, device=dev)
    seq = torch.searchsorted(st["q_start"][1:].long(), row, right=True)
    pos = st["ctx_len"].long()[seq] - st["q_start"].long()[seq + 1] + row
    x = st["qkv"][:tokens].view(tokens, hq + 2 * hkv, D).float()
    cos, sin = (st["cs"][pos][:, None, :, i] for i in (0, 1))
    turn = x[:, :hq + hkv, :rd]
    if case["inter"]:
        a, c = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack([a * cos - c * sin, c * cos + a * sin], dim=-1).flatten(2)
    else:
        a, c = turn[..., :rd // 2], turn[..., rd // 2:]
        turned = torch.cat([a * cos - c * sin, c * cos + a * sin], dim=-1)
    y = torch.cat([turned, x[:, :hq + hkv, rd:]], dim=-1).half()
    st["q_out"][:tokens] = y[:, :hq]
    where = st["table"].long()[seq, pos // page]
    st["k"][where, :, pos % page] = y[:, hq:]
    st["v"][where, :, pos % page] = x[:, hq + hkv:].half()
    return {"q": st["q_out"], "k": st["k"], "v": st["v"]}


def _plain_fork(st):
    kv, table, ctx, refs, src, dst = (st[k] for k in ("kv", "table", "ctx_len", "refs", "src", "dst"))
    page, dev = kv.shape[3], kv.device
    src, dst = src.long(), dst.long()
    place = torch.arange(table.shape[1], device=dev)
    one = torch.ones((), dtype=torch.int32, device=dev)
    # what the targets held goes back
    old = table[dst]
    held = place < (ctx[dst, None] + page - 1) // page
    refs.index_add_(0, old.clamp(min=0).flatten().long(), torch.where(held, -one, 0 * one).flatten())
    # full pages are shared
    n = ctx[src]
    full = place < n[:, None] // page
    rows = table[src]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), torch.where(full, one, 0 * one).flatten())
    new_rows = torch.where(full, rows, -one)
    # the last page, where it is not full, is copied as far as it is filled, to the first free page
    part = torch.nonzero(n % page > 0).flatten()
    new = torch.nonzero(refs == 0).flatten()[:part.numel()]
    last = (n[part] // page).long()
    old_page = rows[part, last].long()
    filled = torch.arange(page, device=dev)[None, :] < (n[part] % page)[:, None]
    kv[:, new] = torch.where(filled[None, :, None, :, None], kv[:, old_page], kv[:, new])
    refs[new] = 1
    new_rows[part, last] = new.int()
    table[dst] = new_rows
    ctx[dst] = n
    st["status"].zero_()
    return {"kv": kv, "table": table, "ctx_len": ctx, "refs": refs, "status": st["status"]}


def _plain_compact(st):
    kv, table, refs, page = st["kv"], st["table"], st["refs"], st["kv"].shape[3]
    refs.copy_(st["refs0"])
    table.copy_(st["table0"])
    n_live = (refs > 0).sum()
    ids = torch.arange(refs.numel(), device=refs.device)
    to = torch.nonzero((refs == 0) & (ids < n_live)).flatten()
    of = torch.nonzero((refs > 0) & (ids >= n_live)).flatten()
    kv[:, to] = kv[:, of]
    refs[to] = refs[of]
    refs[of] = 0
    ids[of] = to
    held = torch.arange(table.shape[1], device=refs.device) < (st["ctx_len"][:, None] + page - 1) // page
    table.copy_(torch.where(held, ids[table.clamp(min=0).long()].int(), table))
    st["n_live"].copy_(n_live.view(1))
    return {"kv": kv, "table": table, "refs": refs, "n_live": st["n_live"]}


def run(st):
    case = st["case"]
    kind = case["kind"]
    if not own:
        return {"attn": _plain_attn, "rope": _plain_rope, "fork": _plain_fork, "compact": _plain_compact}[kind](st)
    import int4_weight_only_02_b200 as i4
    if kind == "attn":
        return i4.paged_gqa_chunk(st["q"], st["k"], st["v"], st["table"], st["q_start"], st["ctx_len"], out=st["out"], window=case["window"],
                                  max_q=st["max_q"], ws=st["ws"])
    if kind == "rope":
        i4.rope_append_chunk(st["qkv"], st["q_start"], st["ctx_len"], st["cs"], case["hq"], case["hkv"], st["k"], st["v"], st["table"],
                             q_out=st["q_out"], interleaved=case["inter"])
        return {"q": st["q_out"], "k": st["k"], "v": st["v"]}
    if kind == "fork":
        i4.kv_pages_fork(st["pools"], st["table"], st["ctx_len"], st["refs"], st["src"], st["dst"], status=st["status"], ws=st["ws"])
        return {"kv": st["kv"], "table": st["table"], "ctx_len": st["ctx_len"], "refs": st["refs"], "status": st["status"]}
    st["refs"].copy_(st["refs0"])
    st["table"].copy_(st["table0"])
    i4.kv_pages_compact(st["pools"], st["table"], st["ctx_len"], st["refs"], n_live=st["n_live"], ws=st["ws"])
    return {"kv": st["kv"], "table": st["table"], "refs": st["refs"], "n_live": st["n_live"]}


# ------------------------------------------------------------------ 64 bits

def _exact_attn(st):
    case = st["case"]
    hq, group, page, window = case["hq"], case["hq"] // case["hkv"], case["page"], case["window"]
    out = torch.zeros((st["q"].shape[0], hq, D), dtype=torch.float64, device=st["q"].device)
    for b, (n, ctx) in enumerate(st["lens"]):
        t = torch.arange(ctx, device=out.device)
        where = st["table"][b].long()[t // page]
        for g in range(case["hkv"]):
            k, v = (st[x][where, g, t % page].double() for x in ("k", "v"))
            for a in range(0, n, 1024):
                e = min(n, a + 1024)
                p = torch.arange(ctx - n + a, ctx - n + e, device=out.device)
                see = (t[None] <= p[:, None]) & ((t[None] > p[:, None] - window) if window else True)
                for h in range(g * group, (g + 1) * group):
                    s = st["q"][st["at"][b] + a:st["at"][b] + e, h].double() @ k.T / math.sqrt(D)
                    s = torch.where(see, s, torch.full_like(s, -math.inf))
                    out[st["at"][b] + a:st["at"][b] + e, h] = torch.exp(s - torch.logsumexp(s, dim=1, keepdim=True)) @ v
    return out


def _exact_rope(st):
    case = st["case"]
    hq, hkv, rd, page = case["hq"], case["hkv"], case["rd"], case["page"]
    scaling, factor, original = _scaling(case)
    f, m = _frequencies(rd, THETA, scaling, factor, original)
    f = torch.tensor(f, dtype=torch.float64, device=st["k"].device)
    q, k, v = st["q_out"].double(), st["k"].double(), st["v"].double()
    first = torch.arange(rd // 2, device=f.device) * (2 if case["inter"] else 1)
    second = first + (1 if case["inter"] else rd // 2)
    for b, (n, ctx) in enumerate(st["lens"]):
        x = st["qkv"][st["at"][b]:st["at"][b] + n].double().view(n, -1, D)
        pos = torch.arange(ctx - n, ctx, device=f.device)
        turn = torch.polar(torch.full((), m, dtype=torch.float64, device=f.device), pos[:, None].double() * f)[:, None]
        z = torch.complex(x[:, :hq + hkv][..., first], x[:, :hq + hkv][..., second]) * turn
        y = x.clone()
        y[:, :hq + hkv, first] = z.real
        y[:, :hq + hkv, second] = z.imag
        where = st["table"][b].long()[pos // page]
        q[st["at"][b]:st["at"][b] + n] = y[:, :hq]
        k[where, :, pos % page] = y[:, hq:hq + hkv]
        v[where, :, pos % page] = y[:, hq + hkv:]
    return {"q": q, "k": k, "v": v}


def _exact_fork(st):
    kv, page = st["kv"].clone(), st["kv"].shape[3]
    table, ctx, refs, src, dst = (st[k].tolist() for k in ("table", "ctx_len", "refs", "src", "dst"))
    for s in dst:
        for p in table[s][:-(-ctx[s] // page)]:
            refs[p] -= 1
        table[s], ctx[s] = [-1] * len(table[s]), 0
    for s, d in zip(src, dst):
        ctx[d] = ctx[s]
        for i in range(ctx[s] // page):
            table[d][i] = table[s][i]
            refs[table[s][i]] += 1
    for s, d in zip(src, dst):
        i, filled = divmod(ctx[s], page)
        if filled:
            new = refs.index(0)
            refs[new], table[d][i] = 1, new
            kv[:, new, :, :filled] = kv[:, table[s][i], :, :filled]
    return {"kv": kv, "table": None, "ctx_len": None, "refs": None, "status": None}


def _exact_compact(st):
    kv, refs = st["kv"].clone(), st["refs0"].tolist()
    n_live = sum(r > 0 for r in refs)
    gaps = [p for p in range(n_live) if refs[p] == 0]
    for to, of in zip(gaps, [p for p in range(n_live, len(refs)) if refs[p] > 0]):
        kv[:, to] = kv[:, of]
    return {"kv": kv, "table": None, "refs": None, "n_live": None}


def exact(case, seed):
    st = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "fork": _exact_fork, "compact": _exact_compact}[case["kind"]](st)
