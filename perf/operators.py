"""The paged KV cache's operators as measured cases: what each call is given,
its plain form, and its definition in 64 bits.

A cache is K and V [n_layers][n_pages][n_kv_heads][page_tokens][head_dim], a
table [n_seqs][max_pages] of page ids (-1: none), the sequences' lengths in
tokens and the pages' reference counts.  Four operators:

  fork       sequences start from the first tokens of others and grow: pages
             are shared, a partly filled page is copied when its sequence grows;
  compact    live pages move to the lowest page ids;
  append     a chunk of new tokens per sequence: QK-norm, rotary positions,
             K and V written into the sequence's pages, q returned;
  attention  a chunk of query rows per sequence over its pages, causal at the
             end of the sequence or (causal = False) over all of it.

Which sequences there are, and how long, follows from the case alone; page
ids and values follow from the seed.
"""
import json
import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-6


# ---- cases -------------------------------------------------------------------

def listed():
    base = dict(layers=1, kv_heads=8, group=2, hd=128, page=16, dtype="fp16")
    return [
        # one short session split into four continuations: the smallest fork
        dict(base, name="fork_small", op="fork", layers=2, kv_heads=2, hd=64, srcs=1, forks=4, tokens=45, grow=1),
        # 32 sessions, eight continuations each, through all 28 layers
        dict(base, name="fork_sessions", op="fork", layers=28, srcs=32, forks=8, tokens=368, grow=12),
        # a small cache closing its gaps
        dict(base, name="compact_small", op="compact", layers=2, kv_heads=2, hd=64, seqs=6, tokens=40, pages=48),
        # a 28-layer cache half full after many sessions have ended
        dict(base, name="compact_store", op="compact", layers=28, seqs=20, tokens=368, pages=1024),
        # one new token in each of eight sequences
        dict(base, name="append_tokens", op="append", seqs=8, rows=1, cached=300, norm=True, rope=True),
        # whole histories of 64 requests written in one call
        dict(base, name="append_histories", op="append", dtype="bf16", page=64, seqs=64, rows=460, cached=32, norm=True,
             rope=True),
        # one token of one request: the smallest attention
        dict(base, name="attend_token", op="attention", seqs=1, rows=1, cached=296, causal=True, lse=False),
        # one token in each of 64 long sequences: K/V bytes
        dict(base, name="attend_long", op="attention", dtype="bf16", page=64, seqs=64, rows=1, cached=16000, causal=True,
             lse=False),
        # new history items of 64 requests over their stored prefixes
        dict(base, name="attend_append", op="attention", seqs=64, rows=36, cached=368, causal=True, lse=False),
        # long chunks over long caches: tensor-core work
        dict(base, name="attend_chunk", op="attention", dtype="bf16", page=128, seqs=4, rows=2048, cached=6144, causal=True,
             lse=False),
        # 256 candidates of 4 tokens per request over the shared prefix, to be joined with their own branches
        dict(base, name="attend_candidates", op="attention", page=32, seqs=16, rows=1024, cached=2132, causal=False,
             lse=True),
        # the fp32 model's cache
        dict(base, name="attend_fp32", op="attention", dtype="fp32", seqs=16, rows=100, cached=1000, causal=True, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = dict(op=rng.choice(["fork", "compact", "append", "attention", "attention", "attention"]), layers=1,
             kv_heads=rng.choice([1, 2, 3, 4, 8]), group=rng.choice([1, 2, 3, 4, 7, 8]), hd=rng.choice([64, 128]),
             page=rng.choice([8, 16, 32, 64, 128]), dtype=rng.choice(["fp16", "fp16", "bf16", "bf16", "fp32"]))
    if c["op"] == "fork":
        c.update(layers=rng.randint(1, 28), srcs=_log(rng, 1, 32), forks=rng.randint(1, 8), tokens=_log(rng, 5, 700),
                 grow=_log(rng, 1, 40))
        limit, size = 2.2e9, lambda: _fork_pages(c) * _page_bytes(c)
    elif c["op"] == "compact":
        c.update(layers=rng.randint(1, 28), seqs=_log(rng, 1, 40), tokens=_log(rng, 5, 700))
        c["pages"] = int(_live_pages(c) * rng.uniform(1.1, 4)) + 2
        limit, size = 1.8e9, lambda: c["pages"] * _page_bytes(c)
    elif c["op"] == "append":
        c.update(seqs=_log(rng, 1, 64), rows=_log(rng, 1, 460), cached=_log(rng, 1, 4000) - 1, norm=rng.random() < 0.8,
                 rope=rng.random() < 0.8)
        limit, size = 4.0e8, lambda: work(c)["bytes"]
    else:
        c.update(seqs=_log(rng, 1, 64), rows=_log(rng, 1, 2048), cached=_log(rng, 1, 16000) - 1, causal=rng.random() < 0.7,
                 lse=rng.random() < 0.5)

        def size():
            n, q, k = c["seqs"], 1.4 * c["rows"], 1.4 * c["cached"] + 1.4 * c["rows"]
            cost = max(work(c)["flops"] * (20 if c["dtype"] == "fp32" else 1) / 4e11, work(c)["bytes"] / 3e9)
            plain = max(n * c["kv_heads"] * c["group"] * q * k * 4 / 4e9, n * c["kv_heads"] * c["hd"] * k * 4 / 6e9)
            return max(cost, plain)
        limit = 1.0
    while size() > limit:  # no more than the largest listed case costs
        k = max((f for f in ("layers", "seqs", "srcs", "rows", "cached") if c.get(f, 0) > 1), key=lambda f: c[f] if f != "layers" else 99)
        c[k] = max(1, int(c[k] * 0.8))
        if c["op"] == "compact":
            c["pages"] = min(c["pages"], 4 * _live_pages(c) + 2)
    return c


def _pages(tokens, page):
    return -(-tokens // page)


def _page_bytes(c):
    return 2 * c["layers"] * c["kv_heads"] * c["page"] * c["hd"] * SIZE[c["dtype"]]


def _ragged(c, tag, n, mean, least=0):
    """n whole numbers around `mean`, the same for every seed."""
    r = random.Random(tag + json.dumps({k: v for k, v in sorted(c.items()) if k not in ("name", "pages")}))
    if mean <= 1 or n == 1:
        return [max(mean, least)] * n
    return [max(least, int(round(mean * r.uniform(0.6, 1.4)))) for _ in range(n)]


def _forks(c):
    """(source lengths, (source, tokens shared, length grown to) of each fork)."""
    lens = _ragged(c, "src", c["srcs"], c["tokens"], 1)
    r = random.Random("fork" + str(c["tokens"]))
    out = []
    for s in range(c["srcs"]):
        for f in range(c["forks"]):
            t = lens[s] if f % 4 != 3 else r.randint(0, lens[s])  # every fourth goes back to an earlier token
            out.append((s, t, t + r.randint(1, c["grow"])))
    return lens, out


def _fork_pages(c):
    lens, forks = _forks(c)
    return sum(_pages(n, c["page"]) for n in lens) + sum(_pages(g, c["page"]) - t // c["page"] for _, t, g in forks) + 3


def _live_pages(c):
    return sum(_pages(n, c["page"]) for n in _ragged(c, "live", c["seqs"], c["tokens"], 1))


def _chunks(c):
    """(rows, whole length) of each sequence of an append or an attention."""
    rows = _ragged(c, "rows", c["seqs"], c["rows"], 1)
    cached = _ragged(c, "cached", c["seqs"], c["cached"])
    if c["op"] == "attention" and not c["causal"]:
        return rows, cached
    return rows, [a + b for a, b in zip(rows, cached)]


# ---- inputs ------------------------------------------------------------------

def _pool(c, n_pages, g):
    shape = (c["layers"], n_pages, c["kv_heads"], c["page"], c["hd"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=DTYPES[c["dtype"]]) for _ in range(2)]


def _table(lens, page, n_pages, max_pages, g):
    """Pages in random order for sequences of these lengths: table, length, refs."""
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    used = (length + page - 1) // page
    col = torch.arange(max_pages, device="cuda")[None]
    first = (torch.cumsum(used, 0) - used)[:, None]
    have = col < used[:, None]
    table = torch.where(have, order[torch.where(have, first + col, 0)], -1).to(torch.int32)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[have].long()] = 1
    return table, length, refs


def _rope_table(positions, hd):
    inv = 1e6 ** (-torch.arange(0, hd // 2, device="cuda", dtype=torch.float64) * 2 / hd)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], -1).float()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) % (1 << 62))
    st = dict(c, status=torch.zeros(4, dtype=torch.int32, device="cuda"))
    if c["op"] == "fork":
        lens, forks = _forks(c)
        n_pages = _fork_pages(c)
        longest = max([_pages(n, c["page"]) for n in lens] + [_pages(f[2], c["page"]) for f in forks])
        st["table"], st["length"], st["refs"] = _table(lens + [0] * len(forks), c["page"], n_pages, longest, g)
        n = c["srcs"]
        st.update(src=_ints([f[0] for f in forks]), dst=_ints([n + i for i in range(len(forks))]),
                  tokens=_ints([f[1] for f in forks]), grown=_ints([f[2] for f in forks]))
    elif c["op"] == "compact":
        lens, n_pages = _ragged(c, "live", c["seqs"], c["tokens"], 1), c["pages"]
        st["table"], st["length"], st["refs"] = _table(lens, c["page"], n_pages, max(_pages(n, c["page"]) for n in lens), g)
        st.update(table_out=torch.empty_like(st["table"]), refs_out=torch.empty_like(st["refs"]),
                  live=torch.empty(1, dtype=torch.int32, device="cuda"))
    else:
        rows, lens = _chunks(c)
        need = sum(_pages(n, c["page"]) for n in lens)
        n_pages = need + 1 + need // 16
        now = [a - b for a, b in zip(lens, rows)] if c["op"] == "append" else lens
        st["table"], st["length"], st["refs"] = _table(now, c["page"], n_pages, max(1, max(_pages(n, c["page"]) for n in lens)), g)
        total, hq, hk = sum(rows), c["kv_heads"] * c["group"], c["kv_heads"]
        # sequences of a batch in an order of their own
        order = torch.randperm(c["seqs"], generator=g, device="cuda")
        st["seq"] = order.to(torch.int32)
        r = torch.tensor(rows, device="cuda")[order]
        st["offset"] = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), torch.cumsum(r, 0)]).to(torch.int32)
        st.update(n_rows=total, max_rows=max(rows), max_len=max(lens))
        if c["op"] == "append":
            st["to"] = torch.tensor(lens, device="cuda")[order].to(torch.int32)
            # the projections' output as one row per token: q, k and v are views of it
            st["qkv"] = torch.randn((total, hq + 2 * hk, c["hd"]), generator=g, device="cuda", dtype=DTYPES[c["dtype"]])
            st["q_gain"], st["k_gain"] = (0.5 + torch.rand(c["hd"], generator=g, device="cuda") for _ in range(2))
            st["rope_table"] = _rope_table(st["max_len"], c["hd"])
            st["q_out"] = torch.empty((total, hq, c["hd"]), device="cuda", dtype=DTYPES[c["dtype"]])
        else:
            st["q"] = torch.randn((total, hq, c["hd"]), generator=g, device="cuda", dtype=DTYPES[c["dtype"]])
            st["out"] = torch.empty_like(st["q"])
            st["lse_out"] = torch.empty((total, hq), device="cuda") if c["lse"] else None
    st["k"], st["v"] = _pool(c, n_pages, g)
    return st


# ---- one pass ----------------------------------------------------------------

def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def _answer(st):
    if st["op"] == "fork":
        return {"table": st["table"], "length": st["length"], "refs": st["refs"], "k": st["k"], "v": st["v"]}
    if st["op"] == "compact":
        return {"table": st["table_out"], "refs": st["refs_out"], "live": st["live"], "k": st["k"], "v": st["v"]}
    if st["op"] == "append":
        return {"q": st["q_out"], "table": st["table"], "length": st["length"], "refs": st["refs"], "k": st["k"],
                "v": st["v"]}
    return {"out": st["out"]} if st["lse_out"] is None else {"out": st["out"], "lse": st["lse_out"]}


def _handles(st, S):
    """The cache and batch objects that a program makes once and keeps."""
    if "cache" not in st:
        ws = torch.empty(S.PagedCache.workspace_bytes(st["k"].shape[1], st["table"].shape[0]), dtype=torch.uint8, device="cuda")
        st["cache"] = S.PagedCache(st["k"], st["v"], st["table"], st["length"], st["refs"], st["status"], ws)
        if "offset" in st:
            hq = st["kv_heads"] * st["group"]
            size = st["cache"].plan_bytes(st["seqs"], st["n_rows"], st["max_rows"], hq)
            st["batch"] = st["cache"].batch(st["seq"], st["offset"], st["n_rows"], st["max_rows"], hq,
                                            torch.empty(size, dtype=torch.uint8, device="cuda"), causal=st.get("causal", True))
    return st["cache"], st.get("batch")


def _own(st):
    import shared_prefix_item_b200 as S
    cache, batch = _handles(st, S)
    stream = torch.cuda.current_stream().cuda_stream
    if st["op"] == "fork":
        cache.free(st["dst"], stream)
        cache.fork(st["src"], st["dst"], st["tokens"], stream)
        cache.resize(st["dst"], st["grown"], stream)
    elif st["op"] == "compact":
        cache.compact(st["table_out"], st["refs_out"], st["live"], stream)
    elif st["op"] == "append":
        hq, hk = st["kv_heads"] * st["group"], st["kv_heads"]
        cache.resize(st["seq"], st["to"], stream)
        batch.plan(stream)
        batch.write(0, st["qkv"][:, :hq], st["qkv"][:, hq:hq + hk], st["qkv"][:, hq + hk:], st["q_out"],
                    q_gain=st["q_gain"] if st["norm"] else None, k_gain=st["k_gain"] if st["norm"] else None, eps=EPS,
                    rope=st["rope_table"] if st["rope"] else None, stream=stream)
    else:
        batch.plan(stream)
        batch.attention(0, st["q"], st["out"], st["lse_out"], st["hd"] ** -0.5, stream)
    return _answer(st)


# ---- plain forms -------------------------------------------------------------

def _plain_resize(st, seq, new):
    page, table, length, refs = st["page"], st["table"], st["length"], st["refs"]
    seq, new = seq.long(), new.long()
    old = length[seq].long()
    p0, p1 = (old + page - 1) // page, (new + page - 1) // page
    tail = table[seq, (p0 - 1).clamp(min=0)].long().clamp(min=0)
    cow = (new > old) & (old % page != 0) & (refs[tail] > 1)
    need = (p1 - p0).clamp(min=0) + cow
    free = torch.cat([(refs == 0).nonzero()[:, 0], torch.zeros(1, dtype=torch.int64, device=refs.device)])
    start = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=table.device)[None]
    rows = table[seq].long()
    fresh = (col >= p0[:, None]) & (col < p1[:, None])
    drop = (col >= p1[:, None]) & (col < p0[:, None])
    refs.index_add_(0, rows[drop], torch.full_like(rows[drop], -1, dtype=torch.int32))
    page_of = free[((start + cow)[:, None] + col - p0[:, None]).clamp(0, free.numel() - 1)]
    rows = torch.where(fresh, page_of, torch.where(drop, -1, rows))
    at, was, now = cow.nonzero()[:, 0], tail[cow], free[start[cow]]
    rows[at, (p0 - 1)[cow]] = now
    refs.index_add_(0, was, torch.full_like(was, -1, dtype=torch.int32))
    refs[rows[fresh]] = 1
    refs[now] = 1
    table[seq] = rows.int()
    length[seq] = new.int()
    keep = (torch.arange(page, device=table.device)[None] < (old % page)[cow][:, None])[None, :, None, :, None]
    for pool in (st["k"], st["v"]):
        pool[:, now] = torch.where(keep, pool[:, was], pool[:, now])


def _plain_fork(st):
    page, table, length, refs = st["page"], st["table"], st["length"], st["refs"]
    src, dst, tokens = st["src"].long(), st["dst"].long(), st["tokens"].long()
    _plain_resize(st, dst, torch.zeros_like(tokens))
    have = torch.arange(table.shape[1], device=table.device)[None] < ((tokens + page - 1) // page)[:, None]
    table[dst] = torch.where(have, table[src], table[dst])
    shared = table[dst][have].long()
    refs.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    length[dst] = tokens.int()
    _plain_resize(st, dst, st["grown"])
    return _answer(st)


def _plain_compact(st):
    refs, table = st["refs"], st["table"]
    live = (refs > 0).sum()
    ids = torch.arange(refs.numel(), device=refs.device)
    src, dst = ((refs > 0) & (ids >= live)).nonzero()[:, 0], ((refs == 0) & (ids < live)).nonzero()[:, 0]
    to = ids.clone()
    to[src] = dst
    have = torch.arange(table.shape[1], device=table.device)[None] < ((st["length"] + st["page"] - 1) // st["page"])[:, None]
    st["table_out"].copy_(torch.where(have, to[table.long().clamp(min=0)], -1))
    st["refs_out"].copy_(torch.where(ids < live, refs, 0))
    st["refs_out"][dst] = refs[src]
    st["live"].copy_(live.reshape(1))
    for pool in (st["k"], st["v"]):
        pool[:, dst] = pool[:, src]
    return _answer(st)


def _rows_of(st):
    """Of each query row: its entry and its position in the sequence."""
    off = st["offset"].long()
    n = off[1:] - off[:-1]
    entry = torch.repeat_interleave(torch.arange(n.numel(), device=off.device), n, output_size=st["n_rows"])
    row = torch.arange(st["n_rows"], device=off.device) - off[entry]
    return entry, st["length"][st["seq"].long()].long()[entry] - n[entry] + row


def _norm_rope(x, gain, rope, pos):
    x = x.float()
    if gain is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gain
    if rope is not None:
        h = x.shape[-1] // 2
        cos, sin = rope[pos][:, None, :, 0], rope[pos][:, None, :, 1]
        x = torch.cat([x[..., :h] * cos - x[..., h:] * sin, x[..., h:] * cos + x[..., :h] * sin], -1)
    return x


def _plain_append(st):
    _plain_resize(st, st["seq"], st["to"])
    hq, hk = st["kv_heads"] * st["group"], st["kv_heads"]
    entry, pos = _rows_of(st)
    page = st["table"][st["seq"].long()[entry], pos // st["page"]].long()
    slot = pos % st["page"]
    rope = st["rope_table"] if st["rope"] else None
    qkv, dt = st["qkv"], st["k"].dtype
    st["q_out"].copy_(_norm_rope(qkv[:, :hq], st["q_gain"] if st["norm"] else None, rope, pos))
    st["k"][0][page, :, slot] = _norm_rope(qkv[:, hq:hq + hk], st["k_gain"] if st["norm"] else None, rope, pos).to(dt)
    st["v"][0][page, :, slot] = qkv[:, hq + hk:]
    return _answer(st)


def _plain_attention(st):
    hk, G, hd, P = st["kv_heads"], st["group"], st["hd"], st["page"]
    off, seq = st["offset"].long(), st["seq"].long()
    n_rows = off[1:] - off[:-1]
    length = st["length"][seq].long()
    n, mq, mp = seq.numel(), st["max_rows"], _pages(st["max_len"], P)
    pages = st["table"][seq, :mp].long().clamp(min=0)
    K, V = (x[0][pages].permute(0, 2, 1, 3, 4).reshape(n, hk, mp * P, hd).float() for x in (st["k"], st["v"]))
    entry, pos = _rows_of(st)
    row = torch.arange(st["n_rows"], device=off.device) - off[entry]
    q = torch.zeros((n, mq, hk, G, hd), device="cuda")
    q[entry, row] = st["q"].float().reshape(-1, hk, G, hd)
    q = q.permute(0, 2, 1, 3, 4).reshape(n, hk, mq * G, hd)
    last = (length - n_rows)[:, None] + torch.arange(mq, device="cuda")[None]  # the last key a row sees
    if not st["causal"]:
        last = (length - 1)[:, None].expand(n, mq)
    hide = torch.arange(mp * P, device="cuda")[None, None] > last[:, :, None]
    s = (q @ K.transpose(-1, -2)).mul_(hd ** -0.5).view(n, hk, mq, G, mp * P)
    s.masked_fill_(hide[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(n, hk, mq * G, mp * P) @ V).view(n, hk, mq, G, hd)
    o = torch.where(total > 0, o / total, 0.0)
    st["out"].copy_(o.permute(0, 2, 1, 3, 4)[entry, row].reshape(-1, hk * G, hd))
    if st["lse_out"] is not None:
        st["lse_out"].copy_((m + total.log()).permute(0, 2, 1, 3, 4)[entry, row].reshape(-1, hk * G))
    return _answer(st)


_PLAIN = {"fork": _plain_fork, "compact": _plain_compact, "append": _plain_append, "attention": _plain_attention}


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    c = case
    es, P, row = SIZE[c["dtype"]], c["page"], 2 * c["layers"] * c["kv_heads"] * c["hd"] * SIZE[c["dtype"]]
    if c["op"] == "fork":
        lens, forks = _forks(c)
        # a partly filled page is read once for all the forks that leave it, and written once by each
        read = {(s, t // P): 0 for s, t, _ in forks}
        wrote = 0
        for s, t, _ in forks:
            read[s, t // P] = max(read[s, t // P], t % P)
            wrote += t % P
        ids = sum(2 * _pages(t, P) + _pages(g, P) for _, t, g in forks)
        return {"bytes": row * (sum(read.values()) + wrote) + 4 * (ids + 4 * len(forks) + 2 * _fork_pages(c)), "flops": 0}
    if c["op"] == "compact":
        live, n = _live_pages(c), c["pages"]
        moved = live * (n - live) / n  # what is expected where pages lie in random order
        table = c["seqs"] * max(_pages(t, P) for t in _ragged(c, "live", c["seqs"], c["tokens"], 1))
        return {"bytes": 2 * moved * row * P + 8 * (table + n), "flops": 0}
    rows, lens = _chunks(c)
    hq, hk, hd, total = c["kv_heads"] * c["group"], c["kv_heads"], c["hd"], sum(rows)
    if c["op"] == "append":
        angles = 4 * hd * max(lens) if c["rope"] else 0
        flops = total * (hq + hk) * hd * ((4 if c["norm"] else 0) + (3 if c["rope"] else 0))
        return {"bytes": 2 * total * (hq + 2 * hk) * hd * es + angles + 8 * sum(_pages(n, P) for n in lens), "flops": flops}
    if c["causal"]:
        pairs = sum(r * (n - r) + r * (r + 1) // 2 for r, n in zip(rows, lens))
    else:
        pairs = sum(r * n for r, n in zip(rows, lens))
    size = 2 * sum(lens) * hk * hd * es + 2 * total * hq * hd * es + (4 * total * hq if c["lse"] else 0)
    return {"bytes": size + 4 * sum(_pages(n, P) for n in lens), "flops": 4 * hd * hq * pairs}


# ---- the definition in 64 bits -----------------------------------------------

class _Book:
    """A cache's tables as lists, changed one sequence at a time."""

    def __init__(self, st):
        self.page = st["page"]
        self.table, self.length, self.refs = st["table"].tolist(), st["length"].tolist(), st["refs"].tolist()
        self.copies = []  # (from page, to page, rows)

    def resize(self, seqs, lengths):
        free = [i for i, r in enumerate(self.refs) if r == 0]
        gone = []
        for s, new in zip(seqs, lengths):
            old, P, row = self.length[s], self.page, self.table[s]
            have, want = -(-old // P), -(-new // P)
            if new > old and old % P and self.shared[row[have - 1]]:
                fresh = free.pop(0)
                self.copies.append((row[have - 1], fresh, old % P))
                gone.append(row[have - 1])
                self.refs[fresh], row[have - 1] = 1, fresh
            for j in range(have, want):
                row[j] = free.pop(0)
                self.refs[row[j]] = 1
            for j in range(want, have):
                gone.append(row[j])
                row[j] = -1
            self.length[s] = new
        for p in gone:
            self.refs[p] -= 1

    def mark(self):
        """Which pages are shared when a call starts."""
        self.shared = [r > 1 for r in self.refs]
        return self

    def fork(self, src, dst, tokens):
        for a, b, t in zip(src, dst, tokens):
            for j in range(-(-t // self.page)):
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            self.length[b] = t


def exact(case, seed):
    st = prepare(case, seed)
    dev = "cuda"
    if st["op"] == "fork":
        b = _Book(st)
        b.fork(st["src"].tolist(), st["dst"].tolist(), st["tokens"].tolist())
        b.mark().resize(st["dst"].tolist(), st["grown"].tolist())
        K, V = st["k"], st["v"]
        for p in (K, V):
            for a, to, rows in b.copies:
                p[:, to, :, :rows] = p[:, a, :, :rows]
        return {"table": torch.tensor(b.table, dtype=torch.int32), "length": torch.tensor(b.length, dtype=torch.int32),
                "refs": torch.tensor(b.refs, dtype=torch.int32), "k": K.double(), "v": V.double()}
    if st["op"] == "compact":
        b = _Book(st)
        n = sum(r > 0 for r in b.refs)
        holes = [i for i in range(n) if b.refs[i] == 0]
        moved = dict(zip([i for i in range(n, len(b.refs)) if b.refs[i]], holes))
        K, V = st["k"], st["v"]
        for p in (K, V):
            for a, to in moved.items():
                p[:, to] = p[:, a]
        for a, to in moved.items():
            b.refs[to], b.refs[a] = b.refs[a], 0
        table = [[moved.get(x, x) for x in row] for row in b.table]
        return {"table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(b.refs, dtype=torch.int32),
                "live": torch.tensor([n], dtype=torch.int32), "k": K.double(), "v": V.double()}
    off, seqs, P, hk, G, hd = st["offset"].tolist(), st["seq"].tolist(), st["page"], st["kv_heads"], st["group"], st["hd"]
    if st["op"] == "append":
        b = _Book(st).mark()
        b.resize(seqs, st["to"].tolist())
        K, V, hq = st["k"].double(), st["v"].double(), hk * G
        x = st["qkv"].double()

        def turned(x, gain, pos):
            if st["norm"]:
                x = x / ((x ** 2).sum(-1, keepdim=True) / hd + EPS).sqrt() * gain.double()
            if st["rope"]:
                t = torch.view_as_complex(st["rope_table"][pos].double().contiguous())[:, None]
                z = torch.complex(x[..., :hd // 2].contiguous(), x[..., hd // 2:].contiguous()) * t
                x = torch.cat([z.real, z.imag], -1)
            return x

        out = torch.empty((st["n_rows"], hq, hd), dtype=torch.float64, device=dev)
        for i, s in enumerate(seqs):
            lo, hi, end = off[i], off[i + 1], b.length[s]
            pos = torch.arange(end - (hi - lo), end, device=dev)
            out[lo:hi] = turned(x[lo:hi, :hq], st["q_gain"], pos)
            at = torch.tensor(b.table[s], device=dev)[pos // P]
            K[0][at, :, pos % P] = turned(x[lo:hi, hq:hq + hk], st["k_gain"], pos)
            V[0][at, :, pos % P] = x[lo:hi, hq + hk:]
        return {"q": out, "table": torch.tensor(b.table, dtype=torch.int32), "length": torch.tensor(b.length, dtype=torch.int32),
                "refs": torch.tensor(b.refs, dtype=torch.int32), "k": K, "v": V}
    out = torch.zeros((st["n_rows"], hk * G, hd), dtype=torch.float64, device=dev)
    lse = torch.full((st["n_rows"], hk * G), -math.inf, dtype=torch.float64, device=dev)
    lens, table = st["length"].tolist(), st["table"].tolist()
    for i, s in enumerate(seqs):
        lo, hi, n = off[i], off[i + 1], lens[s]
        if not n:
            continue
        ids = torch.tensor(table[s][: -(-n // P)], device=dev)
        kv = [x[0].index_select(0, ids).transpose(0, 1).reshape(hk, -1, hd)[:, :n].double() for x in (st["k"], st["v"])]
        for h in range(hk * G):
            s_ = st["q"][lo:hi, h].double() @ kv[0][h // G].T / math.sqrt(hd)
            if st["causal"]:
                s_ = s_ + torch.triu(torch.full_like(s_, -math.inf), diagonal=n - (hi - lo) + 1)
            lse[lo:hi, h] = torch.logsumexp(s_, -1)
            out[lo:hi, h] = torch.softmax(s_, -1) @ kv[1][h // G]
    return {"out": out, "lse": lse} if st["lse"] else {"out": out}
