"""64-bit reference of the softmax layers' operators for long and shared contexts (CPU, torch
float64), and the error bounds of their GPU tests.

Bounds of page keys are values of the cache and a choice of blocks is whole numbers: both are
compared for equality.  Attention over n tokens has the bound that softmax_reference.py derives
(scores: a D-term sum; weights as two bf16 parts; one rounding of the sums per group of 16
tokens, the warps and the pieces); where a shared prefix is streamed in tiles of 128 tokens, the
tensor core adds the 16 products of either part of the weights of a tile, each sum off by at most
2 e of the tile's sum of |p v| (it keeps at least 23 bits), so 32 e for the tile, however many there
are, beside one rounding to nearest a tile.
"""
import math

import torch

import softmax_reference as ref

E = ref.E


def bounds(k_cache, old, block_table, first, seq_lens):
    """The bounds after the new tokens, page by page and token by token."""
    new = old.clone()
    page = k_cache.shape[2]
    most = block_table.shape[1] * page
    for b in range(len(first)):
        n, m = (min(max(int(x[b]), 0), most) for x in (first, seq_lens))
        for i in range(n // page, -(-m // page) if m > n else 0):
            p = int(block_table[b, i])
            if not 0 <= p < k_cache.shape[0]:
                continue
            keys = k_cache[p, :, max(n - i * page, 0):m - i * page]
            lo, hi = keys.amin(1), keys.amax(1)
            if i * page < n:
                lo, hi = torch.minimum(lo, old[p, :, 0]), torch.maximum(hi, old[p, :, 1])
            new[p, :, 0], new[p, :, 1] = lo, hi
    return new


def scores(q, bounds, pages, kv_heads):
    """[Hkv, blocks]: the largest sum of what the bounds allow over a group's heads."""
    h, d = q.shape
    x = bounds[pages.long()].double()  # [blocks, Hkv, 2, d]
    g = q.double().reshape(kv_heads, h // kv_heads, 1, d)
    lo, hi = (x[:, :, i].transpose(0, 1)[:, None] for i in (0, 1))
    s = torch.maximum(g * lo, g * hi).sum(-1)
    return torch.where(torch.isnan(s), math.inf, s).amax(1)


def select(q, bounds_, block_table, seq_lens, page, count, keep_first, keep_last):
    b, kv = q.shape[0], bounds_.shape[1]
    out = torch.full((b, kv, count), -1, dtype=torch.int32)
    for r in range(b):
        n = min(max(int(seq_lens[r]), 0), block_table.shape[1] * page)
        blocks = -(-n // page)
        there = [i for i in range(blocks) if 0 <= int(block_table[r, i]) < bounds_.shape[0]]
        if not there:
            continue
        s = scores(q[r], bounds_, block_table[r, there], kv)
        for j in range(kv):
            kept = [i for i in there if i < keep_first or i >= blocks - keep_last]
            rest = sorted((k for k in range(len(there)) if there[k] not in kept),
                          key=lambda k: (-float(s[j, k]), k))
            got = sorted((kept + [there[k] for k in rest])[:count])
            out[r, j, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def attend(q, k, v, scale, tile=0):
    """q [g, d] over k, v [n, d]: out, lse [g] and the arithmetic parts of their bounds.
    tile: tokens of a tile of the tensor-core path among them (0: none)."""
    q, k, v = q.double(), k.double(), v.double()
    g, d = q.shape
    n = len(k)
    if n == 0:
        z = torch.zeros(g, d, dtype=torch.float64)
        return z, torch.full((g,), -math.inf, dtype=torch.float64), z, torch.zeros(g, dtype=torch.float64)
    s = q @ k.T * scale
    size = (q.abs() @ k.abs().T).amax(1) * abs(scale)
    m = s.amax(1, keepdim=True)
    p = torch.exp(s - m)
    l = p.sum(1, keepdim=True)
    p = p / l
    ds = 2 * E * (d + 8) * size + 8 * E
    factor = 2 * ds + 2.0 ** -16 + 2 * E * (n / 16 + 64) + (32 * E if tile else 0)
    lse = (m + torch.log(l))[:, 0]
    return p @ v, lse, factor[:, None] * (p @ v.abs()), factor + 4 * E * (lse.abs() + m[:, 0].abs() + 1)


def tokens(cache, row, head, n):
    """The first n tokens of a table's row that are there: [m, d]."""
    page = cache.shape[2]
    t = torch.arange(n)
    p = row[t // page].long()
    ok = (p >= 0) & (p < cache.shape[0])
    return cache[p[ok], head, t[ok] % page]


def over(q, parts, scale, tile=0):
    """Attention of every request and head; parts(b, j, cache index) gives the tokens."""
    b, h, d = q.shape
    out, bound = (torch.zeros(b, h, d, dtype=torch.float64) for _ in range(2))
    lse, lbound = (torch.zeros(b, h, dtype=torch.float64) for _ in range(2))
    kv = parts.kv
    for r in range(b):
        for j in range(kv):
            at = slice(j * (h // kv), (j + 1) * (h // kv))
            got = attend(q[r, at], parts(r, j, 0), parts(r, j, 1), scale, tile)
            for x, y in zip((out, lse, bound, lbound), got):
                x[r, at] = y
    return out, lse, bound, lbound


class Chosen:
    """Tokens of chosen blocks: the first min(count, blocks) entries of a row, in their order."""

    def __init__(self, caches, block_table, seq_lens, selected):
        self.caches, self.table, self.lens, self.selected = caches, block_table, seq_lens, selected
        self.kv = caches[0].shape[1]

    def __call__(self, r, j, which):
        cache = self.caches[which]
        page, width = cache.shape[2], self.table.shape[1]
        n = min(max(int(self.lens[r]), 0), width * page)
        blocks = -(-n // page)
        got = []
        for i in self.selected[r, j, :min(self.selected.shape[2], blocks)].tolist():
            if 0 <= i < blocks and 0 <= int(self.table[r, i]) < cache.shape[0]:
                got.append(cache[int(self.table[r, i]), j, :min(page, n - i * page)])
        return torch.cat(got) if got else cache[:0, 0, 0]


class Behind:
    """Tokens of a shared prefix, then the request's own."""

    def __init__(self, caches, prefix_table, prefix_len, block_table, seq_lens):
        self.caches, self.front, self.table, self.lens = caches, prefix_table, block_table, seq_lens
        self.n = min(max(int(prefix_len), 0), len(prefix_table) * caches[0].shape[2])
        self.kv = caches[0].shape[1]

    def __call__(self, r, j, which):
        cache = self.caches[which]
        n = min(max(int(self.lens[r]), 0), self.table.shape[1] * cache.shape[2])
        return torch.cat([tokens(cache, self.front, j, self.n), tokens(cache, self.table[r], j, n)])
