"""A paged cache in plain Python for the tests: its tables as lists changed one
sequence at a time, and its operators in 64 bits."""
import math

import torch

U32 = 2.0 ** -24


def unit(dtype) -> float:
    """Half a step: the largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Book:
    """Tables, lengths and counts as duolm_pages_resize / _fork / _compact leave
    them: free pages are taken lowest first in entry order, and what a call
    gives back is free for later calls only."""

    def __init__(self, n_pages, n_seqs, max_pages, page):
        self.page, self.n_pages = page, n_pages
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.length = [0] * n_seqs
        self.refs = [0] * n_pages

    def pages(self, tokens):
        return -(-tokens // self.page)

    def resize(self, seqs, lengths):
        """The page copies (from, to, rows) of the call."""
        free = [i for i, r in enumerate(self.refs) if r == 0]
        shared = [r > 1 for r in self.refs]
        gone, copies = [], []
        for s, new in zip(seqs, lengths):
            old, row = self.length[s], self.table[s]
            have, want = self.pages(old), self.pages(new)
            if new > old and old % self.page and shared[row[have - 1]]:
                fresh = free.pop(0)
                copies.append((row[have - 1], fresh, old % self.page))
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
        return copies

    def fork(self, src, dst, tokens):
        for a, b, t in zip(src, dst, tokens):
            for j in range(self.pages(t)):
                self.table[b][j] = self.table[a][j]
                self.refs[self.table[a][j]] += 1
            self.length[b] = t

    def compact(self):
        """The moves (from, to) of the call."""
        n = sum(r > 0 for r in self.refs)
        holes = [i for i in range(n) if self.refs[i] == 0]
        moves = dict(zip([i for i in range(n, self.n_pages) if self.refs[i]], holes))
        for a, b in moves.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[moves.get(x, x) if j < self.pages(t) else -1 for j, x in enumerate(row)]
                      for row, t in zip(self.table, self.length)]
        return moves


def rounding(dtype, x):
    """How far one rounding of x to dtype may be off: half a step relative to
    the value, and below the smallest normal value, where the step no longer
    shrinks, half of that fixed step (fp16: 2^-25)."""
    return (unit(dtype) * x.abs()).clamp(min=unit(dtype) * torch.finfo(dtype).smallest_normal) * 1.01


def attention(dtype, q, K, V, scale, rows, length, causal):
    """One entry in 64 bits: q [rows, Hq, hd], K and V [Hkv, length, hd] of the
    sequence, all of dtype.  (out, lse, bound of out, bound of lse).

    Bounds: a score is hd fp32 products and sums, then the scale and the
    exponent's base: ds units of 2^-24, which move a weight and the sum it is
    divided by; the weights are rounded to dtype before they meet V (each by at
    most half a step of a weight, or of the smallest normal one, with the
    largest weight at least 1: their sum is too); exp2 to 2^-22; one fp32
    rounding per key in the sums of the weights and of P V, and 16 for joins;
    last the output's own rounding."""
    q, K, V = q.double(), K.double(), V.double()
    G = q.shape[1] // K.shape[0]
    K, V = K.repeat_interleave(G, 0), V.repeat_interleave(G, 0)
    s = torch.einsum("rhd,hkd->hrk", q, K) * scale
    ds = 0.0
    if length:
        mag = torch.einsum("rhd,hkd->hrk", q.abs(), K.abs()) * scale
        ds = float(((q.shape[2] + 2) * mag + 4 * s.abs()).max())
    if causal:
        last = torch.arange(rows, device=q.device) + length - rows
        s = s.masked_fill(torch.arange(length, device=q.device)[None, None] > last[None, :, None], -math.inf)
    lse = torch.logsumexp(s, -1) if length else torch.full(s.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    p = torch.where(lse[..., None] == -math.inf, 0.0, (s - lse[..., None]).exp())
    out, absv = torch.einsum("hrk,hkd->rhd", p, V), torch.einsum("hrk,hkd->rhd", p, V.abs())
    u = unit(dtype)
    tiny = u * torch.finfo(dtype).smallest_normal * torch.einsum("hrk,hkd->rhd", (s > -math.inf).double(), V.abs())
    bound = rounding(dtype, out) + (u + U32 * (2 * ds + 2 * length + 16 + 8)) * absv + tiny
    lse = lse.transpose(0, 1).contiguous()
    return out, lse, bound, U32 * (2 * ds + length + 32 + 4 * lse.abs())


def norm_rope(x, gain, eps, rope, pos):
    """(values, sum of the magnitudes that make each up) in 64 bits."""
    x = x.double()
    if gain is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * gain.double()
    if rope is None:
        return x, x.abs()
    h = x.shape[-1] // 2
    c, s = rope[pos].double()[:, None, :, 0], rope[pos].double()[:, None, :, 1]
    a, b = x[..., :h], x[..., h:]
    mag = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    return torch.cat([a * c - b * s, b * c + a * s], -1), mag
