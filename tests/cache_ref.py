"""Plain 64-bit references of the operators around the cache, on the CPU, one
sequence and one head at a time, and the inputs their tests share."""

import math

import numpy as np
import torch

HEAD = 64


def tree_words(parents, words):
    """int64 [n, words] ancestor masks of a tree given by parents (-1: a root)."""
    rows = []
    for i, p in enumerate(parents):
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    flat = [[(r >> 64 * w) & 0xFFFFFFFFFFFFFFFF for w in range(words)] for r in rows]
    return torch.from_numpy(np.array(flat, dtype=np.uint64).reshape(len(rows), words).view(np.int64))


def bits(mask_row, n):
    """The first n bits of a row of int64 words."""
    w = mask_row.cpu().numpy().view(np.uint64)
    return np.array([bool(int(w[j // 64]) >> (j % 64) & 1) for j in range(n)], dtype=bool).reshape(n)


class Batch:
    """Sequences over one paged cache: host tensors, with .dev() for the GPU's."""

    def __init__(self, ctx, nodes, H=2, G=4, block_size=16, seed=1, tree=True, words=None, spare=3, q_scale=2.0):
        gen = torch.Generator().manual_seed(seed)
        self.H, self.G, self.bs, self.ctx, self.nodes = H, G, block_size, list(ctx), list(nodes)
        self.B, self.T = len(ctx), sum(nodes)
        counts = [(c + n + block_size - 1) // block_size for c, n in zip(ctx, nodes)]
        self.nb = sum(counts) + spare
        order = torch.randperm(self.nb, generator=gen).to(torch.int32)
        self.tables = torch.full((self.B, max(max(counts), 1)), -7, dtype=torch.int32)
        at = 0
        for b, c in enumerate(counts):
            self.tables[b, :c] = order[at:at + c]
            at += c
        self.cache = torch.randn(self.nb, H, block_size, 2 * HEAD, generator=gen).to(torch.bfloat16)
        self.q = (q_scale * torch.randn(self.T, H * G, HEAD, generator=gen)).to(torch.bfloat16)
        self.ctx_lens = torch.tensor(self.ctx, dtype=torch.int32)
        self.q_starts = torch.tensor(np.concatenate([[0], np.cumsum(nodes)]), dtype=torch.int32)
        self.max_nodes = max(max(nodes), 1)
        self.words = (self.max_nodes + 63) // 64 if words is None else words
        self.mask = None
        if tree:
            rng = np.random.default_rng(seed)
            self.mask = torch.cat([tree_words([int(rng.integers(max(-1, i - 6), i)) if i else -1 for i in range(n)],
                                              self.words) for n in nodes]) if self.T else None

    def cell(self, b, key):
        """(block, page) of a key, or None where there is none."""
        blk = key // self.bs
        if blk >= self.tables.shape[1]:
            return None
        page = int(self.tables[b, blk])
        return None if not 0 <= page < self.nb else (page, key % self.bs)

    def keys(self, b, h, count):
        """K and V [count, 64] in 64 bits (0 where there is none), and which there are."""
        k, v = torch.zeros(count, HEAD, dtype=torch.float64), torch.zeros(count, HEAD, dtype=torch.float64)
        there = np.zeros(count, dtype=bool)
        for j in range(count):
            c = self.cell(b, j)
            if c is not None:
                run = self.cache[c[0], h, c[1]].double()
                k[j], v[j], there[j] = run[:HEAD], run[HEAD:], True
        return k, v, there

    def sees(self, b, there):
        ctx, n = self.ctx[b], self.nodes[b]
        s = np.ones((n, ctx + n), dtype=bool)
        for i in range(n):
            s[i, ctx:] = (np.arange(n) <= i) if self.mask is None else bits(self.mask[int(self.q_starts[b]) + i], n)
        return torch.from_numpy(s & there[None, :])

    def dev(self):
        d = lambda t: None if t is None else t.cuda()
        return dict(q=d(self.q), cache=d(self.cache), tables=d(self.tables), ctx_lens=d(self.ctx_lens),
                    q_starts=d(self.q_starts), tree_mask=d(self.mask), max_nodes=self.max_nodes)


def scores(q, k, scale, cap):
    """(scores, a bound on their error in FP32): sums of 64 exact products,
    each addition within 2^-23 of the sum of magnitudes so far, times scale
    (one rounding, and one of scale log2 e); the cap's own arithmetic adds at
    most 2^-19 of the cap (a handful of operations within 2^-22 on values up to 2)."""
    s = q @ k.T * scale
    err = 64 * 2.0 ** -23 * (q.abs() @ k.abs().T) * scale + s.abs() * 2.0 ** -21
    if cap:
        return cap * torch.tanh(s / cap), err + cap * 2.0 ** -19
    return s, err


def attention(bt, scale=0.125, cap=0.0):
    """(out, lse, bound of out's error, bound of lse's) in 64 bits.

    A weight is off by its score's error e and the exponential's 2^-22
    (relative), and by half a bf16 step (2^-8) in the product with V; the sums of
    N terms by N 2^-24 of their terms' magnitudes, in the numerator and in the
    denominator; out by half a bf16 step of itself. With A = sum p |v| the
    numerator is thus off by (e + 2^-22 + 2^-8 + N 2^-24) A, the
    denominator by (e + 2^-22 + N 2^-24), which moves out by as much of |out| <= A.
    lse is off by log(1 + that) and three roundings of values up to |lse| + 24."""
    T, heads = bt.q.shape[:2]
    out = torch.zeros(T, heads, HEAD, dtype=torch.float64)
    lse = torch.full((T, heads), -math.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(bt.B):
        lo, n = int(bt.q_starts[b]), bt.nodes[b]
        if n == 0:
            continue
        N = bt.ctx[b] + n
        for h in range(bt.H):
            k, v, there = bt.keys(b, h, N)
            sees = bt.sees(b, there)
            for g in range(bt.G):
                hq = h * bt.G + g
                q = bt.q[lo:lo + n, hq].double()
                s, e = scores(q, k, scale, cap)
                for i in range(n):
                    m = sees[i]
                    if not m.any():
                        continue
                    l = torch.logsumexp(s[i][m], 0)
                    p = torch.exp(s[i][m] - l)
                    o, A = p @ v[m], p @ v[m].abs()
                    eps = float(e[i][m].max()) + 2.0 ** -22 + N * 2.0 ** -24
                    out[lo + i, hq], lse[lo + i, hq] = o, l
                    tol_o[lo + i, hq] = o.abs() * 2.0 ** -8 + (2 * eps + 2.0 ** -8) * A * 1.01
                    tol_l[lo + i, hq] = eps * 1.01 + (l.abs() + 24) * 3 * 2.0 ** -24
    return out, lse, tol_o, tol_l


def mass(bt, lse, width, weights=None, decay=1.0, scale=0.125, cap=0.0):
    """(out [B, H, width], bound): a weight e^(s - lse) is off by s's error, three
    roundings of s - lse and the exponential's 2^-22 (relative); the sum over R rows
    by R 2^-24, decay and its addition by 2^-23 of their values."""
    out = torch.zeros(bt.B, bt.H, width, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(bt.B):
        lo, n = int(bt.q_starts[b]), bt.nodes[b]
        N = bt.ctx[b] + n
        W = min(N, width)
        for h in range(bt.H):
            k, _, there = bt.keys(b, h, N)
            if n:
                sees = bt.sees(b, there)
                for g in range(bt.G):
                    hq = h * bt.G + g
                    s, e = scores(bt.q[lo:lo + n, hq].double(), k, scale, cap)
                    live = sees & torch.isfinite(lse[lo:lo + n, hq])[:, None]
                    # (rows that add nothing add no error: 0, not 0 times their infinite difference)
                    d = torch.where(live, s - lse[lo:lo + n, hq].double()[:, None], 0.0)
                    p = torch.where(live, torch.exp(d), 0.0)
                    out[b, h, :W] += p.sum(0)[:W]
                    rel = e + d.abs() * 3 * 2.0 ** -24 + 2.0 ** -22 + n * bt.G * 2.0 ** -24
                    tol[b, h, :W] += (p * rel * 1.01).sum(0)[:W]
            if weights is not None:
                out[b, h, :W] += weights[b, h, :W].double() * decay
            tol[b, h, :W] += out[b, h, :W].abs() * 2.0 ** -22 + 1e-37
    return out, tol


def evict(cache, tables, lens, weights, positions, ends, budget, sinks, recent):
    """The kept cells by a plain sort: (new_weights, new_positions, new_lens, cache)."""
    cache = cache.clone()
    B, H, width = weights.shape
    nb, _, bs, _ = cache.shape
    new_w = torch.zeros(B, H, budget, dtype=torch.float32)
    new_p = torch.full((B, H, budget), -1, dtype=torch.int32)
    new_l = torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        n = max(0, min(int(lens[b]), width, tables.shape[1] * bs))
        kept = min(n, budget)
        new_l[b] = kept
        for h in range(H):
            w, p = weights[b, h, :n].tolist(), positions[b, h, :n].tolist()

            def rank(i):
                x = -math.inf if math.isnan(w[i]) else w[i]
                safe = p[i] < sinks or p[i] >= int(ends[b]) - recent
                return (0, 0.0, i) if safe else (1, -x, i)

            keep = set(sorted(range(n), key=rank)[:kept])
            far = sorted(i for i in keep if i >= kept)
            origin = list(range(kept))
            for to, frm in zip([i for i in range(kept) if i not in keep], far):
                origin[to] = frm
            for to, frm in enumerate(origin):
                new_w[b, h, to], new_p[b, h, to] = weights[b, h, frm], positions[b, h, frm]
                if to == frm:
                    continue
                pt, pf = int(tables[b, to // bs]), int(tables[b, frm // bs])
                if 0 <= pt < nb and 0 <= pf < nb:
                    cache[pt, h, to % bs] = cache[pf, h, frm % bs].clone()
    return new_w, new_p, new_l, cache
