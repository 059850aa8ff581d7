"""The paged cache on the GPU: its tables against the same calls on lists, its
write and attention against 64 bits, with every slot that no sequence owns
holding NaN."""
import math
import random

import pytest

import paged

pytestmark = pytest.mark.gpu

DT = ("fp16", "bf16", "fp32")


def _t():
    import torch
    return torch


def dtype_of(name):
    torch = _t()
    return {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}[name]


def ints(v):
    torch = _t()
    return torch.tensor(v, dtype=torch.int32, device="cuda").reshape(-1)


class Cache:
    """A paged cache with a Book beside it; every slot starts as NaN."""

    def __init__(self, dtype="fp16", layers=1, heads=2, hd=64, page=16, n_pages=64, n_seqs=8, max_pages=16):
        import shared_prefix_item_b200 as S
        torch = _t()
        self.dt = dtype_of(dtype)
        shape = (layers, n_pages, heads, page, hd)
        self.k, self.v = (torch.full(shape, math.nan, dtype=self.dt, device="cuda") for _ in range(2))
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device="cuda")
        self.length = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        ws = torch.full((S.PagedCache.workspace_bytes(n_pages, n_seqs),), 0xA5, dtype=torch.uint8, device="cuda")
        self.c = S.PagedCache(self.k, self.v, self.table, self.length, self.refs, self.status, ws)
        self.book = paged.Book(n_pages, n_seqs, max_pages, page)
        self.page, self.heads, self.hd, self.layers = page, heads, hd, layers

    def same(self):
        self.c.check()
        assert self.table.tolist() == self.book.table
        assert self.length.tolist() == self.book.length
        assert self.refs.tolist() == self.book.refs

    def resize(self, seqs, lengths, stream=None):
        self.c.resize(ints(seqs), ints(lengths), stream)
        return self.book.resize(seqs, lengths)

    def fork(self, src, dst, tokens):
        self.c.fork(ints(src), ints(dst), ints(tokens))
        self.book.fork(src, dst, tokens)

    def free(self, seqs):
        self.c.free(ints(seqs))
        self.book.resize(seqs, [0] * len(seqs))

    def fill(self, g, scale=1.0):
        """Random K and V for every token of every sequence."""
        torch = _t()
        for s, n in enumerate(self.book.length):
            for x in (self.k, self.v):
                for j in range(self.book.pages(n)):
                    m = min(self.page, n - j * self.page)
                    x[:, self.book.table[s][j], :, :m] = (scale * torch.randn((self.layers, self.heads, m, self.hd), generator=g, device="cuda")).to(self.dt)

    def kv(self, layer, s):
        """K and V of a sequence: [heads, length, hd]."""
        torch = _t()
        n = self.book.length[s]
        ids = torch.tensor(self.book.table[s][: self.book.pages(n)], dtype=torch.int64, device="cuda")
        return [x[layer, ids].permute(1, 0, 2, 3).reshape(self.heads, -1, self.hd)[:, :n] for x in (self.k, self.v)]

    def batch(self, seqs, rows, n_q_heads, causal=True, spare=0, max_rows=None):
        torch = _t()
        off = [0]
        for r in rows:
            off.append(off[-1] + r)
        n_rows = off[-1] + spare
        most = max(rows, default=0) if max_rows is None else max_rows
        plan = torch.full((max(128, self.c.plan_bytes(len(seqs), n_rows, most, n_q_heads)),), 0x5A, dtype=torch.uint8, device="cuda")
        return self.c.batch(ints(seqs), ints(off), n_rows, most, n_q_heads, plan, causal=causal), off, n_rows


def gen(seed):
    return _t().Generator(device="cuda").manual_seed(seed)


# ---- tables ------------------------------------------------------------------

@pytest.mark.parametrize("page", [8, 16, 64, 256])
@pytest.mark.parametrize("seed", [1, 2])
def test_random_calls_leave_the_tables_of_the_same_calls_on_lists(page, seed):
    """Resizes, forks, frees and compactions in random order; every sequence
    keeps its own tokens' K and V through all of them."""
    torch = _t()
    r = random.Random(100 * page + seed)
    n_seqs, max_pages = 12, 9
    c = Cache(layers=3, heads=2, hd=64, page=page, n_pages=96, n_seqs=n_seqs, max_pages=max_pages)
    tokens = {s: [] for s in range(n_seqs)}  # what each sequence should hold: one number per token

    def slots(s, lo, hi):
        pos = torch.arange(lo, hi, device="cuda")
        ids = torch.tensor(c.book.table[s], device="cuda")[pos // page]
        return ids, pos % page

    def put(s, lo, hi):
        for t in range(lo, hi):
            tokens[s].append(r.randint(0, 2000))
        ids, sl = slots(s, lo, hi)
        val = torch.tensor(tokens[s][lo:hi], device="cuda", dtype=c.dt)
        c.k[:, ids, :, sl] = val[:, None, None, None].expand(-1, c.layers, c.heads, c.hd)
        c.v[:, ids, :, sl] = -val[:, None, None, None].expand(-1, c.layers, c.heads, c.hd)

    for step in range(25):
        op = r.choice(["resize", "resize", "fork", "free", "compact"])
        if op == "resize":
            seqs = r.sample(range(n_seqs), r.randint(1, 6))
            new = [r.choice([0, 1, page, page + 1, r.randint(0, max_pages * page // 2)]) for _ in seqs]
            old = [c.book.length[s] for s in seqs]
            if sum(c.book.pages(n) + 1 for n in new) > sum(x == 0 for x in c.book.refs):
                continue
            c.resize(seqs, new)
            for s, o, n in zip(seqs, old, new):
                del tokens[s][n:]
                if n > o:
                    put(s, o, n)
        elif op == "fork":
            empty = [s for s in range(n_seqs) if c.book.length[s] == 0]
            full = [s for s in range(n_seqs) if c.book.length[s] > 0]
            if not empty or not full:
                continue
            dst = r.sample(empty, r.randint(1, len(empty)))
            src = [r.choice(full) for _ in dst]
            t = [r.choice([c.book.length[s], r.randint(0, c.book.length[s])]) for s in src]
            c.fork(src, dst, t)
            for a, b, n in zip(src, dst, t):
                tokens[b] = tokens[a][:n]
        elif op == "free":
            seqs = r.sample(range(n_seqs), r.randint(1, 4))
            c.free(seqs)
            for s in seqs:
                tokens[s] = []
        else:
            live = torch.zeros(1, dtype=torch.int32, device="cuda")
            c.c.compact(c.table, c.refs, live)
            c.book.compact()
            assert live.item() == sum(x > 0 for x in c.book.refs)
        c.same()
        for s in range(n_seqs):
            K, V = c.kv(2, s)
            want = torch.tensor(tokens[s], device="cuda", dtype=c.dt)[None, :, None].expand(c.heads, -1, c.hd)
            assert torch.equal(K, want) and torch.equal(V, -want), (step, op, s)


def test_copy_on_write_copies_the_filled_rows_of_every_layer_and_nothing_else():
    torch = _t()
    c = Cache("bf16", layers=2, heads=3, hd=128, page=16, n_pages=16, n_seqs=6, max_pages=4)
    c.resize([0], [21])
    c.fill(gen(1))
    c.fork([0, 0, 0], [1, 2, 3], [21, 21, 18])
    before = c.k.clone(), c.v.clone()
    copies = c.resize([1, 0, 3], [22, 40, 19])  # the source grows too: page 1 is left by all three and stays with 2
    c.same()
    assert len(copies) == 3 and c.book.refs[1] == 1
    for x, was in zip((c.k, c.v), before):
        for a, b, rows in copies:
            was[:, b, :, :rows] = was[:, a, :, :rows]
        assert torch.equal(torch.nan_to_num(x, 7.0), torch.nan_to_num(was, 7.0))


def test_pages_given_back_are_not_taken_by_the_same_call():
    c = Cache(n_pages=4, n_seqs=3, max_pages=4)
    c.resize([0], [32])
    c.resize([0, 1], [1, 32])  # 0 gives back page 1; 1 takes 2 and 3
    c.same()
    assert c.book.table[1][:2] == [2, 3]


def test_compact_into_other_arrays_keeps_the_old_tables_valid():
    torch = _t()
    c = Cache("fp16", layers=2, n_pages=24, n_seqs=4, max_pages=8)
    c.resize([0, 1, 2], [50, 70, 33])
    c.fill(gen(2))
    c.free([0])
    old = [c.kv(l, s) for l in range(2) for s in (1, 2)]
    table, refs = c.table.clone(), c.refs.clone()
    t2, r2, live = torch.full_like(table, 99), torch.full_like(refs, 99), torch.zeros(1, dtype=torch.int32, device="cuda")
    c.c.compact(t2, r2, live)
    c.c.check()
    assert torch.equal(c.table, table) and torch.equal(c.refs, refs)
    assert all(torch.equal(a, b) for x, y in zip(old, [c.kv(l, s) for l in range(2) for s in (1, 2)]) for a, b in zip(x, y))
    moves = c.book.compact()
    assert moves and t2.tolist() == c.book.table and r2.tolist() == c.book.refs and live.item() == 8
    assert all(torch.equal(a, b) for x, y in zip(old, [c.kv(l, s) for l in range(2) for s in (1, 2)]) for a, b in zip(x, y))


def test_compact_of_an_empty_and_of_a_full_cache():
    torch = _t()
    c = Cache(n_pages=4, n_seqs=2, max_pages=4)
    live = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    c.c.compact(c.table, c.refs, live)
    c.same()
    assert live.item() == 0
    c.resize([1], [64])
    c.c.compact(c.table, c.refs, live)
    c.same()
    assert live.item() == 4


def test_many_sequences_and_pages_cross_the_planner_s_blocks():
    """More entries than one block of the scan, and free pages far into the list."""
    c = Cache(layers=1, heads=1, hd=64, page=8, n_pages=9000, n_seqs=3000, max_pages=3)
    r = random.Random(3)
    seqs = list(range(3000))
    r.shuffle(seqs)
    c.resize(seqs, [r.randint(0, 24) for _ in seqs])
    c.same()
    c.free(seqs[::3])
    c.resize(seqs[::2], [r.randint(0, 24) for _ in seqs[::2]])
    c.same()
    live = ints([0])
    c.c.compact(c.table, c.refs, live)
    c.book.compact()
    c.same()


def test_copies_and_moves_of_a_whole_grid():
    """Enough page copies, and then moves, for every SM: what each sequence
    holds is what it held, in every layer."""
    torch = _t()
    c = Cache("bf16", layers=8, heads=4, hd=64, page=16, n_pages=700, n_seqs=80, max_pages=8)
    src = list(range(16))
    c.resize(src, [17 + 5 * i for i in src])
    c.fill(gen(21))
    held = {s: [[x.clone() for x in c.kv(l, s)] for l in range(8)] for s in src}
    dst = list(range(16, 80))
    take = [c.book.length[d % 16] - (d % 3) for d in dst]
    c.fork([d % 16 for d in dst], dst, take)
    copies = c.resize(dst, [t + 3 for t in take])
    assert len(copies) > 50
    c.same()

    def check():
        for s in src + dst:
            n = c.book.length[s] if s in src else take[dst.index(s)]
            for l in range(8):
                for got, want in zip(c.kv(l, s), held[s if s in src else s % 16][l]):
                    assert torch.equal(got[:, :n], want[:, :n]), (s, l)
    check()
    c.free(src[::2] + dst[::3])
    src, gone = src[1::2], set(dst[::3])
    take, dst = [t for t, d in zip(take, dst) if d not in gone], [d for d in dst if d not in gone]
    live = ints([0])
    c.c.compact(c.table, c.refs, live)
    assert c.book.compact()
    c.same()
    check()


# ---- refusals on the device ----------------------------------------------------

def _refused(c, code, call):
    """The call raises the status word and changes nothing; a later call does
    nothing until check() has reported it."""
    import shared_prefix_item_b200 as S
    torch = _t()
    before = [x.clone() for x in (c.table, c.length, c.refs)]
    call()
    c.c.resize(ints([7]), ints([5]))  # skipped
    with pytest.raises(S.DuolmError) as e:
        c.c.check()
    assert e.value.code == code
    assert all(torch.equal(a, b) for a, b in zip(before, (c.table, c.length, c.refs)))
    c.c.check()
    c.same()


@pytest.mark.parametrize("code, seqs, lengths", [
    (-5, [1, 2], [64, 200]), (-5, [0, 1, 2, 3], [256, 256, 256, 17]), (-1, [1, 1], [5, 6]), (-1, [8], [1]), (-1, [-1], [1]),
    (-1, [1], [-1]), (-1, [1], [257])])
def test_a_refused_resize_changes_nothing(code, seqs, lengths):
    c = Cache(n_pages=16, n_seqs=8, max_pages=16)
    c.resize([0, 3], [20, 1])
    _refused(c, code, lambda: c.c.resize(ints(seqs), ints(lengths)))


@pytest.mark.parametrize("src, dst, tokens", [
    ([0], [0], [5]), ([0, 1], [1, 2], [5, 0]), ([0, 0], [1, 1], [5, 5]), ([0], [3], [1]), ([0], [1], [21]), ([0], [1], [-1]),
    ([8], [1], [0]), ([0], [9], [1])])
def test_a_refused_fork_changes_nothing(src, dst, tokens):
    c = Cache(n_pages=16, n_seqs=8, max_pages=16)
    c.resize([0, 3], [20, 1])
    _refused(c, -1, lambda: c.c.fork(ints(src), ints(dst), ints(tokens)))


@pytest.mark.parametrize("seqs, off", [([0, 0], [0, 1, 2]), ([0, 8], [0, 1, 2]), ([0, 3], [0, 2, 1]), ([0, 3], [1, 2, 3]),
                                       ([0, 3], [0, 1, 9])])
def test_a_refused_plan_runs_nothing(seqs, off):
    import shared_prefix_item_b200 as S
    torch = _t()
    c = Cache(n_pages=16, n_seqs=8, max_pages=16)
    c.resize([0, 3], [20, 1])
    c.fill(gen(3))
    b, _, _ = c.batch([0, 3], [2, 1], 4)
    q = torch.randn((3, 4, 64), device="cuda").half()
    out = torch.full_like(q, 5.0)
    bad = c.c.batch(ints(seqs), ints(off), 3, 2, 4, b._arrays[2])

    def call():
        bad.plan()
        bad.attention(0, q, out, None, 0.125)
    _refused(c, -1, call)
    for _ in range(2):  # its plan is refused until the batch is planned again
        bad.attention(0, q, out, None, 0.125)
        with pytest.raises(S.DuolmError) as e:
            c.c.check()
        assert e.value.code == -8
    assert bool((out == 5.0).all())
    b.plan()
    b.attention(0, q, out, None, 0.125)
    c.c.check()
    assert not bool((out == 5.0).any())


def test_a_plan_of_other_sizes_is_refused():
    import shared_prefix_item_b200 as S
    torch = _t()
    c = Cache(n_pages=16, n_seqs=8, max_pages=16)
    c.resize([0, 3], [20, 1])
    c.fill(gen(3))
    q = torch.randn((3, 4, 64), device="cuda").half()
    plan = torch.full((64 << 20,), 0x33, dtype=torch.uint8, device="cuda")
    one = c.c.batch(ints([0, 3]), ints([0, 2, 3]), 3, 2, 4, plan)
    others = [c.c.batch(ints([0, 3]), ints([0, 2, 3]), 3, 2, 4, plan, causal=False),
              c.c.batch(ints([0]), ints([0, 2]), 3, 2, 4, plan), c.c.batch(ints([0, 3]), ints([0, 2, 3]), 3, 9, 4, plan)]

    def refused(b):
        out = torch.full_like(q, 5.0)
        b.attention(0, q, out, None, 0.125)
        with pytest.raises(S.DuolmError) as e:
            c.c.check()
        assert e.value.code == -8 and bool((out == 5.0).all())
    refused(one)  # the buffer holds no plan at all
    one.plan()
    for b in others:
        refused(b)
    out = torch.full_like(q, 5.0)
    one.attention(0, q, out, None, 0.125)
    c.c.check()
    assert not bool((out == 5.0).any())


def test_page_ids_out_of_range_are_reported_not_followed():
    import shared_prefix_item_b200 as S
    torch = _t()
    for dt, rows in (("fp16", 1), ("fp16", 40), ("fp32", 1), ("fp32", 40)):
        c = Cache(dt, n_pages=16, n_seqs=8, max_pages=16)
        c.resize([0], [100])
        c.fill(gen(4))
        b, _, n = c.batch([0], [rows], 4)
        q = torch.randn((n, 4, 64), device="cuda").to(c.dt)
        out = torch.zeros_like(q)
        b.plan()
        c.c.check()
        for bad in (16, -1, 1 << 30, -(1 << 31)):
            was = c.table[0, 2].item()
            c.table[0, 2] = bad
            b.attention(0, q, out, None, 0.125)
            with pytest.raises(S.DuolmError) as e:
                c.c.check()
            assert e.value.code == -7
            c.table[0, 2] = was
            b.plan()
        b.attention(0, q, out, None, 0.125)
        c.c.check()


# ---- write -------------------------------------------------------------------

@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd, heads, group, page, norm, rope, with_q", [
    (128, 8, 2, 16, True, True, True), (64, 3, 7, 8, True, False, True), (128, 1, 1, 64, False, True, True),
    (64, 2, 2, 16, False, False, True), (128, 2, 4, 32, True, True, False)])
def test_write_norm_rotation_and_slots(dt, hd, heads, group, page, norm, rope, with_q):
    _check_write(dt, hd, heads, group, page, norm, rope, with_q, [1, 0, 5, 33], [40, 3, 5, 33])


@pytest.mark.parametrize("hd", [32, 96, 160, 192, 224, 256])
def test_write_fp32_head_dims(hd):
    _check_write("fp32", hd, 2, 2, 16, True, True, True, [3, 20], [3, 50])


def test_write_many_rows():
    _check_write("bf16", 128, 8, 2, 64, True, True, True, [400, 1, 700], [400, 900, 701])


def _check_write(dt, hd, heads, group, page, norm, rope, with_q, rows, lens):
    torch = _t()
    g = gen(hd + heads)
    c = Cache(dt, layers=2, heads=heads, hd=hd, page=page, n_pages=sum(-(-n // page) for n in lens) + 3, n_seqs=6,
              max_pages=max(-(-n // page) for n in lens))
    seqs = [4, 0, 3, 1][: len(rows)]
    c.resize(seqs, lens)
    hq = heads * group
    b, off, n = c.batch(seqs, rows, hq, spare=2)
    qkv = torch.randn((n, hq + 2 * heads, hd), generator=g, device="cuda").to(c.dt)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + heads], qkv[:, hq + heads:]
    gq, gk = (torch.randn(hd, generator=g, device="cuda") for _ in range(2)) if norm else (None, None)
    ang = torch.randn((max(lens), hd // 2), generator=g, device="cuda")
    table = torch.stack([ang.cos(), ang.sin()], -1).contiguous() if rope else None
    q_out = torch.full((n, hq, hd), 3.0, device="cuda", dtype=c.dt)
    was = [c.k.clone(), c.v.clone()]
    b.plan()
    b.write(1, q if with_q else None, k, v, q_out if with_q else None, gq, gk, 1e-6, table)
    c.c.check()
    want_k, want_v = (x.double() for x in was)
    mag_k = torch.zeros_like(want_k)
    for i, s in enumerate(seqs):
        lo, hi = off[i], off[i + 1]
        pos = torch.arange(lens[i] - rows[i], lens[i], device="cuda")
        ids = torch.tensor(c.book.table[s], device="cuda")[pos // page]
        wk, mk = paged.norm_rope(k[lo:hi], gk, 1e-6, table, pos)
        want_k[1, ids, :, pos % page], mag_k[1, ids, :, pos % page] = wk, mk
        want_v[1, ids, :, pos % page] = v[lo:hi].double()
        if with_q:
            wq, mq = paged.norm_rope(q[lo:hi], gq, 1e-6, table, pos)
            # one rounding; in fp32 before it: hd sums under a root, the root, three products, the rotation's two and a sum
            assert bool(((q_out[lo:hi].double() - wq).abs() <= paged.rounding(c.dt, wq) + paged.U32 * (hd / 2 + 10) * mq).all())
    fine = ~torch.isnan(want_k)
    assert torch.equal(fine, ~torch.isnan(c.k))
    off_k = (c.k.double() - want_k).abs()[fine]
    assert bool((off_k <= (paged.rounding(c.dt, want_k) + paged.U32 * (hd / 2 + 10) * mag_k)[fine]).all())
    assert torch.equal(torch.nan_to_num(c.v.double(), 7.0), torch.nan_to_num(want_v, 7.0))  # copied as they are
    assert bool((q_out[off[-1]:] == 3.0).all())  # rows behind the last entry
    if not with_q:
        assert bool((q_out == 3.0).all())


def test_write_in_place_and_refusals():
    import shared_prefix_item_b200 as S
    torch = _t()
    c = Cache("fp16", heads=2, hd=64)
    c.resize([0, 1], [20, 4])
    b, off, n = c.batch([0, 1], [3, 4], 4)
    g = gen(9)
    q, k, v = (torch.randn((n, h, 64), generator=g, device="cuda").half() for h in (4, 2, 2))
    rope = torch.randn((20, 32, 2), generator=g, device="cuda")
    gain = torch.ones(64, device="cuda")
    b.plan()
    out = torch.empty_like(q)
    b.write(0, q, k, v, out, gain, gain, 1e-6, rope)
    b.write(0, q, k, v, q, gain, gain, 1e-6, rope)  # q in place
    c.c.check()
    assert torch.equal(q, out)
    b.write(0, None, k, v, None, rope=rope[:19].contiguous())  # position 19 is not in it
    with pytest.raises(S.DuolmError) as e:
        c.c.check()
    assert e.value.code == -1
    more, _, n = c.batch([1], [5], 4)  # five rows of a sequence of four
    more.plan()
    more.write(0, None, k[:5].contiguous(), v[:5].contiguous(), None)
    with pytest.raises(S.DuolmError) as e:
        c.c.check()
    assert e.value.code == -1
    for bad in (dict(k=k.float()), dict(k=k[:3]), dict(v=v.transpose(0, 1)), dict(rope=rope[:, :5]), dict(q_gain=gain.half()),
                dict(k=k.cpu())):
        a = dict(q=q, k=k, v=v, q_out=out)
        a.update(bad)
        with pytest.raises(ValueError):
            b.write(0, **a)


# ---- attention ---------------------------------------------------------------

def _check_attention(dt, hd, heads, group, page, rows, lens, causal=True, spread=1.0, flat=False, seed=0, max_rows=None,
                     layers=1):
    torch = _t()
    g = gen(seed + hd + 7 * heads)
    need = sum(-(-n // page) for n in lens) + 2
    c = Cache(dt, layers=layers, heads=heads, hd=hd, page=page, n_pages=need, n_seqs=len(lens) + 1,
              max_pages=max(1, max(-(-n // page) for n in lens)))
    seqs = list(range(len(lens)))
    random.Random(seed).shuffle(seqs)
    # taken one page at a time in turn, so that a sequence's pages are apart
    for part in range(1, 5):
        c.resize(seqs, [n * part // 4 for n in lens])
    c.fill(g)
    hq, layer = heads * group, layers - 1
    b, off, n = c.batch(seqs, rows, hq, causal=causal, spare=3, max_rows=max_rows)
    wide = (spread * torch.randn((n, hq + 2, hd), generator=g, device="cuda")).to(c.dt)
    q = wide[:, 1:1 + hq] if not flat else wide[:, :hq].reshape(n, hq * hd)
    buf = torch.full((n, hq + 1, hd), 9.0, device="cuda", dtype=c.dt)
    out = buf[:, :hq]
    lse = torch.full((n, hq), 9.0, device="cuda")
    scale = hd ** -0.5
    b.plan()
    b.attention(layer, q, out, lse, scale)
    c.c.check()
    first, first_lse = buf.clone(), lse.clone()
    for i, s in enumerate(seqs):
        lo, hi = off[i], off[i + 1]
        if lo == hi:
            continue
        K, V = c.kv(layer, s)
        qi = q[lo:hi].reshape(hi - lo, hq, hd)
        want, wl, bound, tol = paged.attention(c.dt, qi, K, V, scale, hi - lo, lens[i], causal)
        err = (out[lo:hi].double() - want).abs()
        assert bool((err <= bound).all()), (i, rows[i], lens[i], float((err - bound).max()), float(err.max()))
        none = wl == -math.inf
        assert torch.equal(none, lse[lo:hi] == -math.inf)
        assert bool((out[lo:hi][none] == 0).all())
        assert bool(((lse[lo:hi].double() - wl)[~none].abs() <= tol[~none]).all())
    assert bool((out[off[-1]:] == 9.0).all()) and bool((buf[:, hq:] == 9.0).all()) and bool((lse[off[-1]:] == 9.0).all())
    # again, without the sums: the same bits, whichever CTA came last
    b.attention(layer, q, out, None, scale)
    c.c.check()
    assert torch.equal(buf, first) and torch.equal(lse, first_lse)


LENS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd, heads, group, page", [(128, 8, 2, 16), (64, 2, 7, 8), (128, 1, 16, 64), (64, 3, 1, 256),
                                                    (128, 2, 4, 128), (128, 1, 8, 32)])
def test_attention_of_single_tokens(dt, hd, heads, group, page):
    _check_attention(dt, hd, heads, group, page, [1] * len(LENS), LENS)


@pytest.mark.parametrize("dt", DT)
def test_attention_of_a_few_tokens_each(dt):
    _check_attention(dt, 128, 2, 2, 16, [1, 2, 3, 4, 5, 6, 7, 8, 0, 3], [1, 2, 5, 100, 64, 700, 129, 8, 40, 128])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd, heads, group, page", [(128, 2, 2, 16), (64, 2, 1, 8), (64, 1, 7, 64), (128, 1, 4, 256),
                                                    (128, 1, 64, 32), (64, 2, 3, 128), (128, 2, 5, 8)])
def test_attention_of_chunks(dt, hd, heads, group, page):
    _check_attention(dt, hd, heads, group, page, [1, 5, 64, 65, 130, 0, 200, 33], [1, 5, 100, 65, 513, 7, 200, 1000])


@pytest.mark.parametrize("dt", DT)
def test_attention_of_rows_that_see_nothing(dt):
    """More rows than tokens, and empty sequences: zeros and -infinity."""
    _check_attention(dt, 128, 2, 2, 16, [1, 9, 40, 2, 130], [0, 3, 17, 2, 1])
    _check_attention(dt, 64, 2, 2, 16, [1, 1], [0, 1])
    _check_attention(dt, 64, 2, 2, 16, [3, 70], [0, 0], causal=False)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("hd, heads, group, page", [(128, 2, 2, 32), (64, 2, 5, 16)])
def test_attention_over_whole_sequences(dt, hd, heads, group, page):
    _check_attention(dt, hd, heads, group, page, [1, 300, 4, 64, 2, 17], [77, 129, 0, 640, 1, 64], causal=False)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 3, 100])
def test_attention_divides_a_long_sequence_among_the_ctas(dt, rows):
    _check_attention(dt, 128, 1, 2, 64, [rows], [20011])
    _check_attention(dt, 64, 2, 2, 16, [rows, rows], [4097, 128], seed=1)


@pytest.mark.parametrize("dt", DT)
def test_attention_with_sharp_scores(dt):
    """Scores of some hundreds: one key takes all the weight, and the running
    maximum moves by far more than any fixed range."""
    _check_attention(dt, 128, 2, 2, 16, [1, 70, 150], [500, 333, 150], spread=12.0)
    _check_attention(dt, 128, 2, 2, 16, [1, 2, 1], [500, 333, 1500], spread=12.0)


@pytest.mark.parametrize("dt", DT)
def test_attention_of_a_larger_entry_than_said(dt):
    """max_rows chooses the kernel; an entry with more rows is still right."""
    _check_attention(dt, 128, 2, 2, 16, [50, 1, 9], [70, 90, 300], max_rows=1)
    _check_attention(dt, 64, 2, 2, 16, [3, 1], [70, 90], max_rows=900)


@pytest.mark.parametrize("dt", DT)
def test_attention_of_flat_rows_and_another_layer(dt):
    _check_attention(dt, 64, 2, 2, 16, [1, 40], [70, 90], flat=True, layers=3)
    _check_attention(dt, 128, 2, 2, 16, [1, 2], [70, 90], flat=True, layers=2)


@pytest.mark.parametrize("dt", DT)
def test_attention_of_rows_aligned_to_16_bytes_alone(dt):
    torch = _t()
    g = gen(31)
    c = Cache(dt, heads=1, hd=64, n_pages=40, n_seqs=2, max_pages=20)
    c.resize([1, 0], [300, 70])
    c.fill(g)
    e = 16 // c.k.element_size()
    for rows in ([150, 70], [2, 1]):
        b, off, n = c.batch([1, 0], rows, 2)
        b.plan()
        wide = torch.randn((n, 128 + e), generator=g, device="cuda").to(c.dt)
        buf = torch.full((n, 128 + e), 9.0, device="cuda", dtype=c.dt)
        q, out = wide[:, e:], buf[:, e:]
        b.attention(0, q, out, None, 0.125)
        c.c.check()
        assert bool((buf[:, :e] == 9.0).all())
        for i, s in enumerate([1, 0]):
            want, _, bound, _ = paged.attention(c.dt, q[off[i]:off[i + 1]].reshape(-1, 2, 64), *c.kv(0, s), 0.125, rows[i],
                                                c.book.length[s], True)
            assert bool(((out[off[i]:off[i + 1]].reshape(-1, 2, 64).double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dt, layers", [("fp16", 24), ("fp32", 12)])
def test_a_cache_whose_offsets_pass_32_bits(dt, layers):
    """The last pages of the last layer: more than 2^32 bytes (and, in 16 bits,
    2^31 elements) into K and V."""
    torch = _t()
    g = gen(51)
    heads, hd, page, n_pages, group = 8, 128, 64, 2048, 2
    c = Cache(dt, layers=layers, heads=heads, hd=hd, page=page, n_pages=n_pages, n_seqs=4, max_pages=n_pages)
    c.resize([0], [2030 * page])  # takes the low pages; nothing is written there
    c.resize([1], [300])
    assert min(x for x in c.book.table[1] if x >= 0) == 2030
    last = layers - 1
    for x in (c.k, c.v):
        for j in range(5):
            m = min(page, 300 - page * j)
            x[:, c.book.table[1][j], :, :m] = torch.randn((layers, heads, m, hd), generator=g, device="cuda").to(c.dt)
    held = [x.clone() for x in c.kv(last, 1)]
    c.fork([1], [2], [300])
    c.resize([2], [304])  # a copy of the last page, in every layer
    c.same()
    for rows in (1, 4, 40):
        new = max(0, rows - 4)
        c.resize([2], [304 + new])
        b, off, n = c.batch([2], [rows], heads * group)
        q, k, v = (torch.randn((n, h, hd), generator=g, device="cuda").to(c.dt) for h in (heads * group, heads, heads))
        out = torch.empty_like(q)
        b.plan()
        b.write(last, None, k, v, None)
        if rows >= 4:  # (one row of the four that grew: the others are still NaN)
            b.attention(last, q, out, None, hd ** -0.5)
            K, V = c.kv(last, 2)
            want, _, bound, _ = paged.attention(c.dt, q, K, V, hd ** -0.5, rows, 304 + new, True)
            assert bool(((out.double() - want).abs() <= bound).all())
        c.c.check()
        K, V = c.kv(last, 2)
        assert torch.equal(K[:, -rows:].transpose(0, 1), k) and torch.equal(V[:, -rows:].transpose(0, 1), v)
        assert torch.equal(K[:, :300], held[0]) and torch.equal(V[:, :300], held[1])
    c.free([0])
    live = ints([0])
    c.c.compact(c.table, c.refs, live)
    assert c.book.compact()
    c.same()
    K, V = c.kv(last, 1)
    assert torch.equal(K, held[0]) and torch.equal(V, held[1])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 64])
def test_attention_of_more_tiles_than_are_taken_by_the_unit(dt, rows):
    """Long enough for the CTAs' shares to be cut tile by tile."""
    _check_attention(dt, 64, 4, 2, 64, [rows] * 16, [9000 + 37 * i for i in range(16)])


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 9])
def test_attention_of_more_entries_than_one_cta_plans(dt, rows):
    r = random.Random(7)
    n = 1500
    _check_attention(dt, 64, 1, 2, 8, [r.choice([0, 1, rows, rows]) for _ in range(n)], [r.randint(0, 60) for _ in range(n)],
                     max_rows=rows)


@pytest.mark.parametrize("hd", [32, 96, 160, 192, 224, 256])
def test_attention_fp32_head_dims(hd):
    _check_attention("fp32", hd, 2, 2, 16, [1, 40, 70], [70, 90, 300])
    _check_attention("fp32", hd, 2, 2, 16, [1, 2], [70, 300])


@pytest.mark.parametrize("dt", DT)
def test_attention_of_many_sequences(dt):
    r = random.Random(5)
    n = 300
    _check_attention(dt, 64, 2, 2, 8, [r.choice([0, 1, 1, 2, 40]) for _ in range(n)], [r.randint(0, 200) for _ in range(n)])


def test_attention_arguments_are_checked():
    torch = _t()
    c = Cache("fp16")
    c.resize([0], [20])
    b, _, n = c.batch([0], [3], 4)
    q = torch.zeros((n, 4, 64), device="cuda", dtype=torch.float16)
    lse = torch.zeros((n, 4), device="cuda")
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:2]), dict(out=q.transpose(0, 1)), dict(out=q[..., ::2]),
                dict(lse=lse.half()), dict(lse=lse[:2]), dict(lse=lse.t())):
        a = dict(q=q, out=torch.empty_like(q), lse=lse)
        a.update(bad)
        with pytest.raises(ValueError):
            b.attention(0, a["q"], a["out"], a["lse"], 0.125)


# ---- as they are used together -------------------------------------------------

@pytest.mark.parametrize("dt", DT)
def test_a_session_is_stored_forked_continued_and_compacted(dt):
    """History written in two chunks, forked into candidates' continuations,
    each extended by its own tokens and attended; then the finished ones are
    freed, the rest compacted, and attention gives the same bits."""
    torch = _t()
    g = gen(11)
    heads, group, hd, page, layers = 2, 2, 128, 16, 2
    hq = heads * group
    c = Cache(dt, layers=layers, heads=heads, hd=hd, page=page, n_pages=80, n_seqs=8, max_pages=12)
    gain = 0.5 + torch.rand(hd, generator=g, device="cuda")
    ang = torch.randn((192, hd // 2), generator=g, device="cuda")
    rope = torch.stack([ang.cos(), ang.sin()], -1).contiguous()
    held = {}  # per (layer, sequence): K and V in the cache's dtype, from the written ones

    def append(seqs, rows):
        old = [c.book.length[s] for s in seqs]
        c.resize(seqs, [o + r for o, r in zip(old, rows)])
        b, off, n = c.batch(seqs, rows, hq)
        b.plan()
        outs = []
        for l in range(layers):
            q, k, v = (torch.randn((n, h, hd), generator=g, device="cuda").to(c.dt) for h in (hq, heads, heads))
            out = torch.empty_like(q)
            b.write(l, q, k, v, q, gain, gain, 1e-6, rope)
            b.attention(l, q, out, None, hd ** -0.5)
            for i, s in enumerate(seqs):
                K, V = c.kv(l, s)
                if (l, s) in held:  # what was there before is there still
                    assert torch.equal(K[:, : old[i]], held[l, s][0]) and torch.equal(V[:, : old[i]], held[l, s][1])
                assert not bool(torch.isnan(K).any()) and not bool(torch.isnan(V).any())
                held[l, s] = (K.clone(), V.clone())
                want, _, bound, _ = paged.attention(c.dt, q[off[i]:off[i + 1]], K, V, hd ** -0.5, rows[i], old[i] + rows[i], True)
                assert bool(((out[off[i]:off[i + 1]].double() - want).abs() <= bound).all())
            outs.append((b, l, q, out))
        c.same()
        return outs

    append([6], [40])
    append([0, 1], [70, 33])
    append([1, 0], [20, 9])
    dst = [2, 3, 4, 5]
    c.fork([0, 0, 1, 0], dst, [79, 79, 53, 64])
    for d, s, t in zip(dst, [0, 0, 1, 0], [79, 79, 53, 64]):
        for l in range(layers):
            held[l, d] = tuple(x[:, :t].clone() for x in held[l, s])
    append([5, 3, 2, 0, 4], [3, 1, 40, 2, 20])
    last = append([2, 3, 5, 1], [1, 1, 1, 1])
    c.free([6, 0, 4])
    live = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.c.compact(c.table, c.refs, live)
    assert c.book.compact()
    c.same()
    for b, l, q, out in last:
        again = torch.empty_like(out)
        b.attention(l, q, again, None, hd ** -0.5)
        c.c.check()
        assert torch.equal(again, out)


@pytest.mark.parametrize("dt", DT)
@pytest.mark.parametrize("rows", [1, 40])
def test_a_captured_step_goes_on_as_the_lengths_do(dt, rows):
    """resize, plan, write and attention captured once and replayed with other
    lengths and values, eager calls in between."""
    torch = _t()
    g = gen(12)
    heads, hq, hd = 2, 4, 128
    c = Cache(dt, heads=heads, hd=hd, n_pages=64, n_seqs=4, max_pages=32)
    to, seqs = ints([rows, rows]), [2, 0]
    b, off, n = c.batch(seqs, [rows, rows], hq)
    q, k, v = (torch.zeros((n, h, hd), device="cuda", dtype=c.dt) for h in (hq, heads, heads))
    out = torch.zeros_like(q)
    sq = ints(seqs)

    def step(stream):
        c.c.resize(sq, to, stream)
        b.plan(stream)
        b.write(0, None, k, v, None, stream=stream)
        b.attention(0, q, out, None, hd ** -0.5, stream)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        side.synchronize()
        c.book.resize(seqs, [rows, rows])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(side.cuda_stream)
    for lens in ([rows, rows], [rows + 3, rows + 90], [2 * rows + 50, rows + 100], [rows + 200, 2 * rows + 101]):
        # the sequences' earlier tokens, written eagerly
        c.resize(seqs, lens)
        c.fill(g)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        to.copy_(ints(lens))
        out.zero_()
        graph.replay()
        c.same()
        for i, s in enumerate(seqs):
            lo, hi = off[i], off[i + 1]
            K, V = c.kv(0, s)
            assert torch.equal(K[:, lens[i] - rows:].transpose(0, 1), k[lo:hi])
            want, _, bound, _ = paged.attention(c.dt, q[lo:hi], K, V, hd ** -0.5, rows, lens[i], True)
            assert bool(((out[lo:hi].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("layers", [1, 6])
def test_a_captured_fork_and_compaction(layers):
    """free, fork, resize and compact captured once, replayed over other lengths
    (one layer: a cluster of CTAs; six: a whole grid)."""
    torch = _t()
    n = 24
    c = Cache("fp16", layers=layers, heads=4, hd=64, page=8, n_pages=600, n_seqs=2 * n, max_pages=12)
    src, dst = list(range(n)), list(range(n, 2 * n))
    s_src, s_dst, take, grown, live = ints(src), ints(dst), ints([0] * n), ints([1] * n), ints([0])
    c.resize(src, [5] * n)
    side = torch.cuda.Stream()

    def step(stream):
        c.c.free(s_dst, stream)
        c.c.fork(s_src, s_dst, take, stream)
        c.c.resize(s_dst, grown, stream)
        c.c.compact(c.table, c.refs, live, stream)

    def book(t, g):
        c.book.resize(dst, [0] * n)
        c.book.fork(src, dst, t)
        c.book.resize(dst, g)
        c.book.compact()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(side.cuda_stream)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(side.cuda_stream)
    book([0] * n, [1] * n)
    r = random.Random(layers)
    for _ in range(4):
        c.resize(src, [r.randint(1, 60) for _ in src])
        c.fill(gen(41))
        held = [[x.clone() for x in c.kv(layers - 1, s)] for s in src]
        t = [r.randint(0, c.book.length[s]) for s in src]
        g = [x + r.randint(0, 20) for x in t]
        take.copy_(ints(t))
        grown.copy_(ints(g))
        graph.replay()
        book(t, g)
        c.same()
        for i in range(n):
            for got, src_kv, want in zip(c.kv(layers - 1, dst[i]), c.kv(layers - 1, src[i]), held[i]):
                assert torch.equal(got[:, : t[i]], want[:, : t[i]]) and torch.equal(src_kv, want)


def test_calls_follow_their_stream():
    """A step on a side stream, behind work that the stream still has to do."""
    torch = _t()
    c = Cache("fp16", heads=2, hd=64, n_pages=64, n_seqs=4, max_pages=32)
    side = torch.cuda.Stream()
    k = torch.randn((300, 2, 64), device="cuda").half()
    q = torch.randn((300, 4, 64), device="cuda").half()
    late = torch.zeros_like(k)
    out = torch.zeros_like(q)
    b, _, _ = c.batch([1], [300], 4)
    big = torch.randn((4096, 4096), device="cuda")
    seqs, lens = ints([1]), ints([300])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big = big @ big * 1e-3
        late.copy_(k)
        s = side.cuda_stream
        c.c.resize(seqs, lens, s)
        b.plan(s)
        b.write(0, None, late, late, None, stream=s)
        b.attention(0, q, out, None, 0.125, s)
    c.c.check(s)
    c.book.resize([1], [300])
    c.same()
    K, V = c.kv(0, 1)
    assert torch.equal(K.transpose(0, 1), k)
    want, _, bound, _ = paged.attention(c.dt, q, K, V, 0.125, 300, 300, True)
    assert bool(((out.double() - want).abs() <= bound).all())
