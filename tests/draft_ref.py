"""Plain 64-bit references of the operators on a drafted token's way to the cache
and over it, with the bounds on the kernels' errors."""

import torch


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def halves(x, R, layout):
    return (x[..., 0:R:2], x[..., 1:R:2]) if layout == "interleaved" else (x[..., :R // 2], x[..., R // 2:R])


def turn(x, pos, table, layout, sign=1.0):
    """(x turned, the sum of the magnitudes of each element's terms)."""
    R = table.shape[1]
    row = table.double()[pos][:, None, :]
    c, s = row[..., :R // 2], row[..., R // 2:] * sign
    out, size = x.clone(), x.abs()
    a, b = halves(x, R, layout)
    oa, ob = halves(out, R, layout)
    sa, sb = halves(size, R, layout)
    oa.copy_(a * c - b * s), ob.copy_(b * c + a * s)
    sa.copy_((a * c).abs() + (b * s).abs()), sb.copy_((b * c).abs() + (a * s).abs())
    return out, size


def norm_rotate(x, w, pos, table, layout, eps):
    """(y, bound). In FP32 the sum of d squares is off by d 2^-24 of itself, the mean, eps and 1 / sqrt by
    four roundings, and the root halves what the sum brings: with x r and times w (two roundings) and the turn's
    product and FMA n is off by (d / 2 + 8) 2^-24 of its terms; then half a step of the type (a subnormal's:
    half of the least value)."""
    d, dt = x.shape[-1], x.dtype
    x = x.double()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        n = n * w.double()
    y, size = turn(n, pos, table, layout)
    tol = size * (d / 2 + 8) * 2.0 ** -24 * 1.01 + y.abs() * half_step(dt) * 1.01
    return y, tol + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def norm_rotate_grad(gy, x, w, pos, table, layout, eps):
    """(dx, its bound, dw, its bound). With e = (d / 2 + 8) 2^-24 for x r: g is off by 2 2^-24 of its terms
    G, a product g w x r by e + 4 2^-24 of G |w x r|, their mean by d 2^-24 more, dx by the sum of those times r
    and half a step. dw sums N such products: N 2^-24 of their magnitudes, and half a step of the gains' type."""
    T, H, d = x.shape
    dt = x.dtype
    x, gy = x.double(), gy.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    u = x * r
    g, G = turn(gy, pos, table, layout, -1.0)
    gain = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    along = (g * gain * u).mean(-1, keepdim=True)
    dx = r * (g * gain - u * along)
    e = (d / 2 + 8) * 2.0 ** -24
    mean = (G * gain.abs() * u.abs()).mean(-1, keepdim=True)
    tol = r * (G * gain.abs() * (e + 6 * 2.0 ** -24) + u.abs() * mean * (3 * e + (d + 8) * 2.0 ** -24)) * 1.01
    tol = tol + dx.abs() * half_step(dt) * 1.01 + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    dw = (g * u).sum((0, 1))
    wt = torch.float32 if w is None else w.dtype
    dw_tol = (G * u.abs()).sum((0, 1)) * (e + (T * H + 6) * 2.0 ** -24) * 1.01 + dw.abs() * half_step(wt) * 1.01
    return dx, tol, dw, dw_tol + torch.finfo(wt).smallest_normal * torch.finfo(wt).eps


STEPS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def fp4_groups(x):
    """[..., 32] -> (code numbers, exponents) by the definition, element by element in 64 bits: the least e in -120 ..
    125 with which the largest is at most 6 2^e (125 at the most), and the nearest value, of two the even code."""
    x = x.double()
    most = x.abs().amax(-1)
    e = torch.full(most.shape, -120, dtype=torch.int64)
    for _ in range(246):
        e = torch.where((most > 6 * torch.exp2(e.double())) & (e < 125), e + 1, e)
    y = x.abs() * torch.exp2(-e.double())[..., None]  # (exact: a power of two)
    far = torch.stack([(y - s).abs() for s in STEPS], -1)
    least = far.amin(-1, keepdim=True)
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])  # even codes first
    code = order[(far[..., order] == least).to(torch.int8).argmax(-1)]
    return code, e


def fp4_values(x):
    """What a [..., 64] row of K or V stands for once stored."""
    g = x.double().unflatten(-1, (2, 32))
    code, e = fp4_groups(g)
    sign = torch.where(torch.signbit(g), -1.0, 1.0)
    return (torch.tensor(STEPS, dtype=torch.float64)[code] * sign * torch.exp2(e.double())[..., None]).flatten(-2)


def make_batch():
    """cache_ref.Batch with a window and sinks, and (after pack) with the values of a cache of 4 bits."""
    import numpy as np

    from cache_ref import Batch, bits

    class WindowBatch(Batch):
        window, sinks = None, 0

        def behind(self, window, sinks=0):
            self.window, self.sinks = window, sinks
            return self

        def sees(self, b, there):
            s = super().sees(b, there).numpy().copy()
            if self.window is None:
                return torch.from_numpy(s)
            ctx, n, lo = self.ctx[b], self.nodes[b], int(self.q_starts[b])
            key = np.arange(ctx + n)
            for i in range(n):
                if self.mask is None:
                    s[i] &= (key < self.sinks) | (key > ctx + i - self.window)
                else:
                    p = ctx + int(bits(self.mask[lo + i], n).sum()) - 1
                    s[i, :ctx] &= ((key < self.sinks) | (key > p - self.window))[:ctx]
            return torch.from_numpy(s)

        def pack(self, nrc, fill=0xFF):
            """The cache as cells of 4 bits on the GPU (bytes of no cell: fill); its values become the reference's cache."""
            page = nrc.fp4_page_bytes(self.bs)
            packed = torch.full((self.nb, self.H, page), fill, dtype=torch.uint8, device="cuda")
            rows = self.cache.transpose(1, 2).reshape(-1, self.H, 128).cuda()
            slots = torch.arange(self.nb * self.bs, device="cuda")
            nrc.context_fp4_store(rows[..., :64], rows[..., 64:], slots, packed)
            k, v = nrc.context_fp4_load(packed, slots)
            self.cache = torch.cat([k, v], -1).unflatten(0, (self.nb, self.bs)).transpose(1, 2).cpu()
            return packed

        def wipe(self, packed, b, key, byte=None, gen=None):
            """A key's cell filled with one byte, or with random ones."""
            block, at = self.cell(b, key)
            for first, width in ((0, 32), (32 * self.bs, 32), (64 * self.bs, 4)):
                run = packed[block, :, first + at * width:first + (at + 1) * width]
                run.copy_(torch.randint(0, 256, run.shape, generator=gen).to(torch.uint8) if byte is None
                          else torch.full_like(run, byte))

    return WindowBatch


def dense_attention(bt, scale=0.125):
    """cache_ref.attention of chains behind bt's window (None: none), all rows of a head at once, on the GPU in 64 bits
    (for rows and keys too many to go through one by one): (out, lse, bound of out's error, bound of lse's)."""
    dev = "cuda"
    T, heads = bt.q.shape[:2]
    out = torch.zeros(T, heads, 64, dtype=torch.float64, device=dev)
    lse = torch.full((T, heads), -torch.inf, dtype=torch.float64, device=dev)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    q, cache, tables = bt.q.to(dev), bt.cache.to(dev), bt.tables.to(dev).long()
    for b in range(bt.B):
        lo, n, ctx = int(bt.q_starts[b]), bt.nodes[b], bt.ctx[b]
        key = torch.arange(ctx + n, device=dev)
        block = key // bt.bs
        page = tables[b][block.clamp(max=tables.shape[1] - 1)]
        there = (block < tables.shape[1]) & (page >= 0) & (page < bt.nb)
        own = ctx + torch.arange(n, device=dev)[:, None]
        sees = there & (key <= own)
        if bt.window is not None:
            sees &= (key < bt.sinks) | (key > own - bt.window)
        sees = sees.repeat_interleave(bt.G, 0)
        for h in range(bt.H):
            kv = cache[page.clamp(0, bt.nb - 1), h, key % bt.bs].double() * there[:, None]
            k, v = kv[:, :64], kv[:, 64:]
            of = slice(h * bt.G, (h + 1) * bt.G)
            x = q[lo:lo + n, of].double().flatten(0, 1)
            s = x @ k.T * scale
            e = 64 * 2.0 ** -23 * (x.abs() @ k.abs().T) * scale + s.abs() * 2.0 ** -21
            s = s.masked_fill(~sees, -torch.inf)
            l = torch.logsumexp(s, 1)
            some = l > -torch.inf
            p = torch.exp(s - torch.where(some, l, 0.0)[:, None])
            o, A = p @ v, p @ v.abs()
            eps = e.masked_fill(~sees, 0.0).amax(1) + 2.0 ** -22 + (ctx + n) * 2.0 ** -24
            fold = lambda t: t.unflatten(0, (n, bt.G))
            out[lo:lo + n, of], lse[lo:lo + n, of] = fold(o), fold(l)
            tol_o[lo:lo + n, of] = fold(o.abs() * 2.0 ** -8 + (2 * eps[:, None] + 2.0 ** -8) * A * 1.01)
            tol_l[lo:lo + n, of] = fold(torch.where(some, eps * 1.01 + (l.abs() + 24) * 3 * 2.0 ** -24, 0.0))
    return out, lse, tol_o, tol_l


def sum_depth(T, heads, others, lanes, num_cus):
    """How many additions a term of the gains' gradients passes at most: the heads of T rows go two (or one) a group of `lanes` lanes, to
    workgroups of 256 / lanes groups, 8 a CU that the queries and keys (heads and others) share; a lane adds its group's
    rounds, a workgroup its groups, the joining launch's threads a 64th of the workgroups each in four sums (and up to three
    more in the first), then these, then 64 threads' by halves."""
    groups, pairs, other_pairs = 256 // lanes, T * (-(-heads // 2)), T * (-(-others // 2))
    most = 8 * num_cus
    blocks = min(-(-pairs // groups), max(1, most * pairs // (pairs + other_pairs) - 1))
    return 2 * -(-pairs // (blocks * groups)) + groups + blocks // 256 + 4 + 2 + 6


def gains_grad(gy, x, w, pos, table, layout, eps, depth):
    """(dw, its bound) of norm_rotate_grad by the depth of the sums, which is far less than the number of their terms: with e = (d
    / 2 + 8) 2^-24 for x r a term g x r is off by e + 4 2^-24 of G |x r|, each addition that it passes adds 2^-24 of it, and
    the sum is rounded to the gains' type."""
    d = x.shape[-1]
    x, gy = x.double(), gy.double()
    u = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    g, G = turn(gy, pos, table, layout, -1.0)
    dw = (g * u).sum((0, 1))
    tol = (G * u.abs()).sum((0, 1)) * (d / 2 + 12 + depth) * 2.0 ** -24 * 1.01 + dw.abs() * half_step(w.dtype) * 1.01
    return dw, tol + torch.finfo(w.dtype).smallest_normal * torch.finfo(w.dtype).eps
