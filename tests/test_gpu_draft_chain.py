"""The operators on a drafted token's way to the cache run together, captured, at
their largest sizes and offsets."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from draft_ref import fp4_values, norm_rotate  # noqa: E402


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def exact(q, k, v, table, bs, ctx, n, rows, window=None, sinks=0, mask=None):
    """(out, lse, sum of p |v|) in 64 bits of rows `rows` of one sequence's nodes on one KV head; k, v: [blocks, bs, 64]."""
    key = torch.arange(ctx + n, device=q.device)
    page = table.long()[key // bs]
    k, v = k[page, key % bs].double(), v[page, key % bs].double()
    s = q.double() @ k.T.contiguous() / 8.0
    sees = key[None] <= ctx + rows[:, None] if mask is None else torch.cat([torch.ones(len(rows), ctx, dtype=torch.bool, device=q.device), mask], 1)
    if window is not None:
        sees = sees & ((key[None] < sinks) | (key[None] > ctx + rows[:, None] - window))
    s = s.masked_fill(~sees, -math.inf)
    l = torch.logsumexp(s, 1)
    p = torch.exp(s - l[:, None])
    return p @ v, l, p @ v.abs()


def near(out, lse, want, terms, most):
    """The bounds of cache_ref.attention, with the scores' error bounded by that of the largest sum of magnitudes `most`."""
    o, l, A = want
    eps = 64 * 2.0 ** -23 * most + 2.0 ** -22 + terms * 2.0 ** -24
    assert bool(((out.double() - o).abs() <= o.abs() * 2.0 ** -8 + (2 * eps + 2.0 ** -8) * A * 1.01 + 1e-30).all())
    assert bool(((lse.double() - l).abs() <= eps * 1.01 + (l.abs() + 24) * 3 * 2.0 ** -24).all())


def magnitude(q, k):
    """The largest sum of |q_i k_i| / 8 that a score can have."""
    return float(q.double().norm(dim=-1).max() * k.double().norm(dim=-1).max()) / 8


def test_from_the_projection_to_the_attention(nrc):
    """Two layers: the projection's rows normed and turned, stored in 4 bits, attended to; each step against its own
    definition, the attention also against the bf16 attention over the same values; then all of it captured."""
    gen = torch.Generator().manual_seed(1)
    L, T, H, G, bs, D, ctx = 2, 40, 2, 4, 16, 8192, 23
    normed = torch.randn(L, T, D, generator=gen).bfloat16().cuda()
    w = (torch.randn(L, D, 2 * H * 64, generator=gen) / 90).bfloat16().cuda()
    kv = nrc.context_kv_project(normed, w)
    pos = torch.randperm(500, generator=gen)[:T].cuda()
    cs = nrc.rope_table(500, 64, dtype=torch.float32)
    gain = (1 + 0.2 * torch.randn(64, generator=gen)).bfloat16().cuda()
    blocks = 9
    order = torch.randperm(blocks, generator=gen)[:3].int()
    slots = (order.long()[torch.arange(T) // bs] * bs + torch.arange(T) % bs).cuda()
    tables = order[None].cuda()
    q = torch.randn(T - ctx, H * G, 64, generator=gen).bfloat16().cuda()
    qpos = pos[ctx:].contiguous()
    lens = torch.tensor([ctx], dtype=torch.int32).cuda()
    starts = torch.tensor([0, T - ctx], dtype=torch.int32).cuda()
    caches = torch.zeros(L, blocks, H, nrc.fp4_page_bytes(bs), dtype=torch.uint8, device="cuda")

    def step():
        k, v = nrc.kv_views(kv, H)
        q1 = nrc.qk_norm_rotate(q, None, qpos, cs, gain)[0]
        keys = torch.stack([nrc.qk_norm_rotate(k[l], None, pos, cs, eps=1e-6)[0] for l in range(L)])
        nrc.context_fp4_store(keys, v, slots, caches)
        outs = [nrc.context_fp4_attention(q1, caches[l], tables, lens, starts, T - ctx, window=30, sinks=2) for l in range(L)]
        return [q1, keys] + [t for o in outs for t in o]

    got = step()
    k, v = nrc.kv_views(kv, H)
    for x, y, g, p in ((q, got[0], gain, qpos), (k[0], got[1][0], None, pos), (k[1], got[1][1], None, pos)):
        want, tol = norm_rotate(x.cpu(), None if g is None else g.cpu(), p.cpu(), cs.cpu(), "interleaved", 1e-6)
        assert bool(((y.double().cpu() - want).abs() <= tol).all())
    lk, lv = nrc.context_fp4_load(caches, slots)
    assert torch.equal(lk.double().cpu(), fp4_values(got[1].cpu())) and torch.equal(lv.double().cpu(), fp4_values(v.cpu()))
    for l in range(L):
        plain = torch.zeros(blocks, H, bs, 128, dtype=torch.bfloat16, device="cuda")
        plain[slots // bs, :, slots % bs] = torch.cat([lk[l], lv[l]], -1)
        o, s = nrc.context_window_attention(got[0], plain, tables, lens, starts, T - ctx, 30, 2)
        A = lv[l].abs().max()
        # the same keys, values and formula, summed in another order: each within its bound, twice (2^-8 a weight and half a step of out)
        assert bool(((got[2 + 2 * l].float() - o.float()).abs() <= 4 * 2.0 ** -8 * A).all())
        assert bool(((got[3 + 2 * l] - s).abs() <= 1e-4 + s.abs() * 2.0 ** -20).all())
        most = magnitude(got[0], lk[l])
        rows = torch.arange(T - ctx, device="cuda")
        for h in range(H):
            for g in range(G):
                want = exact(got[0][:, h * G + g], plain[:, h, :, :64], plain[:, h, :, 64:], order.cuda(), bs, ctx, T - ctx, rows, 30, 2)
                near(got[2 + 2 * l][:, h * G + g], got[3 + 2 * l][:, h * G + g], want, T, most)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        for t in held:
            t.zero_()
        caches.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, got))
        step()


@pytest.mark.parametrize("fp4", [False, True])
def test_offsets_past_32_bits(nrc, fp4):
    """Caches past 2^32 bytes (and elements), pages at their far ends, few rows and many."""
    bs, H, ctx = 16, 4, 700
    page = nrc.fp4_page_bytes(bs)
    blocks = (1 << 32) // (H * page) + 2000 if fp4 else (1 << 32) // (H * bs * 128) + 2000
    gen = torch.Generator().manual_seed(2)
    for n, G in ((2, 4), (40, 4)):
        table = (blocks - 1 - torch.randperm(1500, generator=gen)[:50]).int()
        table[::3] = torch.randperm(1000, generator=gen)[:17].int()
        kv = torch.randn(50 * bs, H, 128, generator=gen).bfloat16().cuda()
        slots = (table.long()[:, None] * bs + torch.arange(bs)).flatten().cuda()
        q = torch.randn(n, H * G, 64, generator=gen).bfloat16().cuda()
        args = dict(tables=table[None].cuda(), ctx_lens=torch.tensor([ctx], dtype=torch.int32).cuda(),
                    q_starts=torch.tensor([0, n], dtype=torch.int32).cuda(), max_nodes=n, window=600, sinks=3)
        if fp4:
            cache = torch.empty(blocks, H, page, dtype=torch.uint8, device="cuda")
            nrc.context_fp4_store(kv[..., :64], kv[..., 64:], slots, cache)
            k, v = nrc.context_fp4_load(cache, slots)
            assert torch.equal(k.double().cpu(), fp4_values(kv[..., :64].cpu()))
            out, lse = nrc.context_fp4_attention(q, cache, **args)
        else:
            cache = torch.empty(blocks, H, bs, 128, dtype=torch.bfloat16, device="cuda")
            cache[slots // bs, :, slots % bs] = kv
            k, v = kv[..., :64], kv[..., 64:]
            out, lse = nrc.context_window_attention(q, cache, **args)
        rows, local = torch.arange(n, device="cuda"), torch.arange(50, device="cuda")
        for hq in range(H * G):
            h = hq // G
            want = exact(q[:, hq], k[:, h].unflatten(0, (50, bs)), v[:, h].unflatten(0, (50, bs)), local, bs, ctx, n, rows, 600, 3)
            near(out[:, hq], lse[:, hq], want, ctx + n, magnitude(q, k))
        del cache


@pytest.mark.parametrize("fp4", [False, True])
def test_the_longest_chain(nrc, fp4):
    """65535 nodes behind a window (and, packed, a chain of 20000 without one), sampled rows."""
    n, window, sinks, bs, ctx = 65535, 100, 6, 16, 50
    if fp4:
        n, window = 20000, None
    gen = torch.Generator().manual_seed(3)
    blocks = (ctx + n + bs - 1) // bs
    table = torch.randperm(blocks, generator=gen).int().cuda()
    cache = torch.randn(blocks, 1, bs, 128, generator=gen).bfloat16().cuda()
    q = torch.randn(n, 2, 64, generator=gen).bfloat16().cuda()
    args = dict(tables=table[None], ctx_lens=torch.tensor([ctx], dtype=torch.int32).cuda(),
                q_starts=torch.tensor([0, n], dtype=torch.int32).cuda(), max_nodes=n, window=window or 0, sinks=sinks)
    if fp4:
        packed = torch.empty(blocks, 1, nrc.fp4_page_bytes(bs), dtype=torch.uint8, device="cuda")
        slots = torch.arange(blocks * bs, device="cuda")
        rows = cache.transpose(1, 2).reshape(-1, 1, 128)
        nrc.context_fp4_store(rows[..., :64], rows[..., 64:], slots, packed)
        k, v = (t.view(blocks, bs, 64) for t in nrc.context_fp4_load(packed, slots))
        out, lse = nrc.context_fp4_attention(q, packed, **args)
    else:
        k, v = cache[:, 0, :, :64], cache[:, 0, :, 64:]
        out, lse = nrc.context_window_attention(q, cache, **args)
    rows = torch.cat([torch.arange(260), torch.randint(0, n, (200,), generator=gen), torch.arange(n - 260, n)]).cuda()
    for h in range(2):
        want = exact(q[rows, h], k, v, table, bs, ctx, n, rows, window, sinks)
        near(out[rows, h], lse[rows, h], want, ctx + n if fp4 else window + sinks, magnitude(q, k))


@pytest.mark.parametrize("B,H,nodes,G", [(100, 1, 5, 8), (130, 2, 9, 4), (300, 1, 1, 40), (70, 1, 3, 4), (2, 2, 48, 8)])
def test_ragged_batches(nrc, B, H, nodes, G):
    """Packed caches of many sequences of very different lengths (some empty), whose shares follow the lengths."""
    gen = torch.Generator().manual_seed(B)
    bs = 16
    ctx = [int(3000 * 1.5 ** -float(torch.rand(1, generator=gen) * 20)) for _ in range(B)]
    counts = [int(torch.randint(0 if b % 7 == 3 else 1, nodes + 1, (1,), generator=gen)) for b in range(B)]
    need = [(c + n + bs - 1) // bs for c, n in zip(ctx, counts)]
    order = torch.randperm(sum(need) + 3, generator=gen).int()
    tables, at = torch.full((B, max(need)), -1, dtype=torch.int32), 0
    for b, c in enumerate(need):
        tables[b, :c] = order[at:at + c]
        at += c
    blocks = len(order)
    rows = torch.randn(blocks * bs, H, 128, generator=gen).bfloat16().cuda()
    packed = torch.full((blocks, H, nrc.fp4_page_bytes(bs)), 0xFF, dtype=torch.uint8, device="cuda")
    slots = torch.arange(blocks * bs, device="cuda")
    nrc.context_fp4_store(rows[..., :64], rows[..., 64:], slots, packed)
    k, v = (t.view(blocks, bs, H, 64) for t in nrc.context_fp4_load(packed, slots))
    starts = torch.tensor([0] + counts).cumsum(0).int()
    q = torch.randn(int(starts[-1]), H * G, 64, generator=gen).bfloat16().cuda()
    out, lse = nrc.context_fp4_attention(q, packed, tables.cuda(), torch.tensor(ctx, dtype=torch.int32).cuda(), starts.cuda(),
                                         max(max(counts), 1))
    most = magnitude(q, k)
    for b in range(B):
        lo, n = int(starts[b]), counts[b]
        if n == 0:
            continue
        for hq in range(H * G):
            want = exact(q[lo:lo + n, hq], k[:, :, hq // G], v[:, :, hq // G], tables[b].cuda(), bs, ctx[b], n,
                         torch.arange(n, device="cuda"))
            near(out[lo:lo + n, hq], lse[lo:lo + n, hq], want, ctx[b] + n, most)


def test_calls_at_once(nrc):
    """Two streams, each with operands and results of its own, many calls on the way together."""
    gen = torch.Generator().manual_seed(4)
    sets = []
    for i in range(2):
        kv = torch.randn(600, 2, 128, generator=gen).bfloat16().cuda()
        packed = torch.zeros(40, 2, nrc.fp4_page_bytes(16), dtype=torch.uint8, device="cuda")
        slots = torch.randperm(640, generator=gen)[:600].cuda()
        q = torch.randn(12, 8, 64, generator=gen).bfloat16().cuda()
        sets.append((kv, packed, slots, q, torch.arange(40, dtype=torch.int32).cuda()[None],
                     torch.tensor([500 + 20 * i], dtype=torch.int32).cuda(), torch.tensor([0, 12], dtype=torch.int32).cuda()))

    def step(s, stream=None):
        kv, packed, slots, q, tables, lens, starts = s
        nrc.context_fp4_store(kv[..., :64], kv[..., 64:], slots, packed, stream=stream)
        return nrc.context_fp4_attention(q, packed, tables, lens, starts, 12, stream=stream)

    want = [step(s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    got = [[step(s, st) for s, st in zip(sets, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in got:
        for g, w in zip(pair, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_a_captured_training_step(nrc):
    """Forward and backward with gains captured and replayed on new inputs; a second derivative raises instead of being
    silently incomplete."""
    gen = torch.Generator().manual_seed(5)
    new = lambda *shape: torch.randn(*shape, generator=gen).bfloat16().cuda()
    T, cs, pos = 70, nrc.rope_table(100, 64), torch.arange(70).cuda()
    q, k, qw, kw, gq, gk = new(T, 8, 64), new(T, 2, 64), new(64), new(64), new(T, 8, 64), new(T, 2, 64)

    def step():
        leaves = [t.detach().requires_grad_() for t in (q, k, qw, kw)]
        outs = nrc.qk_norm_rotate(leaves[0], leaves[1], pos, cs, leaves[2], leaves[3])
        return [t.detach() for t in outs] + list(torch.autograd.grad(outs, leaves, [gq, gk]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for _ in range(3):
        q.copy_(new(T, 8, 64)), gk.copy_(new(T, 2, 64)), qw.copy_(new(64))
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))
    leaf = q.float().requires_grad_()
    out, _ = nrc.qk_norm_rotate(leaf, None, pos, cs)
    grad, = torch.autograd.grad(out.square().sum(), leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.sum().backward()
