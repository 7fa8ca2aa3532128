"""The operators around the cache run as they are used: table, store, rotated
queries, attention, received weights, eviction, and decoding on what is left."""

import pytest

import cache_ref as ref
from helpers import to_host
from test_gpu_tree_attention import assert_within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


I32 = dict(dtype=torch.int32)


def slots_of(bt, b, first, count):
    return [int(bt.tables[b, j // bt.bs]) * bt.bs + j % bt.bs for j in range(first, first + count)]


def test_store_attend_weigh_evict_and_decode(nrc):
    """Two layers; contexts stored, a drafted tree attended and weighed, its accepted path's cells evicted down to a
    budget, then single tokens on the smaller cache with an eviction after each."""
    H, G, L, budget, recent, sinks = 2, 4, 2, 64, 8, 4
    bt = ref.Batch([100, 45, 70], [6, 9, 3], H=H, G=G, seed=31)
    gen = torch.Generator().manual_seed(32)
    table = nrc.rope_table(400, 64, scaling="ramp", factor=4.0, original_max=100, magnitude=1.1)
    assert table.shape == (400, 64)
    caches = torch.zeros(L, bt.nb, H, bt.bs, 128, dtype=torch.bfloat16, device="cuda")
    tables = bt.tables.cuda()

    def store(rows):
        """rows: (sequence, cell, position); random K and V of every layer."""
        kv = torch.randn(L, len(rows), 2 * H * 64, generator=gen).to(torch.bfloat16).cuda()
        slots = torch.tensor([slots_of(bt, b, c, 1)[0] for b, c, _ in rows], device="cuda")
        nrc.context_kv_store(kv, torch.tensor([p for _, _, p in rows], device="cuda"), slots, table, caches, H)

    store([(b, j, j) for b in range(3) for j in range(bt.ctx[b] + bt.nodes[b])])
    lens, ends = list(bt.ctx), [c + n for c, n in zip(bt.ctx, bt.nodes)]
    state = [None] * L  # weights and positions of the cells, by layer
    for step in range(4):
        nodes = bt.nodes if step == 0 else [1, 1, 1]
        bt.ctx, bt.nodes, bt.T = list(lens), list(nodes), sum(nodes)
        if step:
            store([(b, lens[b], ends[b]) for b in range(3)])
            ends = [e + 1 for e in ends]
            bt.mask = None
            bt.q_starts = torch.tensor([0, 1, 2, 3], **I32)
        positions = torch.tensor([ends[b] - nodes[b] + i for b in range(3) for i in range(nodes[b])])
        cells = [n + k for n, k in zip(lens, nodes)]
        width = max(cells)
        d = dict(ctx=torch.tensor(lens, **I32).cuda(), starts=bt.q_starts.cuda(), lens=torch.tensor(cells, **I32).cuda(),
                 ends=torch.tensor(ends, **I32).cuda(), mask=None if bt.mask is None else bt.mask.cuda())
        for layer in range(L):
            raw = (2 * torch.randn(bt.T, H * G, 64, generator=gen)).to(torch.bfloat16).cuda()
            q = nrc.rope_rotate(raw, positions.cuda(), table)
            bt.q, bt.cache = q.cpu(), caches[layer].cpu()
            args = (q, caches[layer], tables, d["ctx"], d["starts"])
            out, lse = nrc.context_tree_attention(*args, max(nodes), tree_mask=d["mask"])
            o, l, to, tl = ref.attention(bt)
            assert_within(out, o, to, f"out of step {step}, layer {layer}")
            assert_within(lse, l, tl, f"lse of step {step}, layer {layer}")
            old_w = torch.zeros(3, H, width)
            pos = torch.zeros(3, H, width, **I32)
            for b in range(3):
                n = lens[b]
                if state[layer] is None:
                    pos[b, :, :n] = torch.arange(n)
                else:
                    old_w[b, :, :n], pos[b, :, :n] = state[layer][0][b, :, :n], state[layer][1][b, :, :n]
                pos[b, :, n:n + nodes[b]] = torch.arange(ends[b] - nodes[b], ends[b])
            w = nrc.context_attention_mass(*args, lse, max(nodes), tree_mask=d["mask"], weights=old_w.cuda(), decay=0.9,
                                           width=width)
            want, tol = ref.mass(bt, lse.cpu(), width, old_w, 0.9)
            assert_within(w, want, tol, f"weights of step {step}, layer {layer}")
            got = nrc.context_kv_evict(caches[layer], tables, d["lens"], w, pos.cuda(), d["ends"], budget, sinks, recent)
            want = ref.evict(bt.cache, bt.tables, d["lens"].cpu(), w.cpu(), pos, d["ends"].cpu(), budget, sinks, recent)
            for g, x in zip(got, want):
                assert torch.equal(g.cpu(), x)
            assert (to_host(caches[layer]) == to_host(want[3])).all()
            state[layer] = (got[0].cpu(), got[1].cpu())
        lens = got[2].tolist()
        assert lens == [min(c, budget) for c in cells]


def test_captured_step_follows_the_lengths(nrc):
    """One captured step (attention, weights, eviction) replayed while the lengths on the device grow."""
    H, G, budget = 2, 4, 200
    for nodes in (1, 40):  # few rows, many rows
        bt = ref.Batch([1100, 1100], [nodes, nodes], H=H, G=G, seed=33, tree=False)
        d = bt.dev()
        gen = torch.Generator().manual_seed(34)
        w = torch.rand(2, H, 1200, generator=gen).cuda()
        p = torch.arange(1200, **I32).expand(2, H, 1200).contiguous().cuda()
        lens = torch.tensor([1100, 1100], **I32).cuda()

        def step(cache, ctx):
            out, lse = nrc.context_tree_attention(d["q"], cache, d["tables"], ctx, d["q_starts"], nodes, max_ctx=1100)
            m = nrc.context_attention_mass(d["q"], cache, d["tables"], ctx, d["q_starts"], lse, nodes, max_ctx=1100,
                                           weights=w, decay=0.5)
            return (out, lse, m, *nrc.context_kv_evict(cache, d["tables"], ctx + nodes, m, p, ctx + nodes, budget, 4, 16))

        step(d["cache"].clone(), lens)
        torch.cuda.synchronize()
        cache = d["cache"].clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(cache, lens)
        for n in ([3, 0], [64, 700], [1100, 1], [600, 1100]):
            lens.copy_(torch.tensor(n, **I32))
            cache.copy_(d["cache"])
            for o in outs:
                o.fill_(1)
            g.replay()
            eager_cache = d["cache"].clone()
            eager = step(eager_cache, lens)
            torch.cuda.synchronize()
            for a, b in zip(outs, eager):
                assert torch.equal(a, b)
            assert torch.equal(cache.view(torch.int16), eager_cache.view(torch.int16))


def test_blocks_of_a_shared_prefix(nrc):
    """Sequences whose tables begin with the same blocks, and one block twice in a table."""
    bt = ref.Batch([80, 90, 50], [5, 20, 1], H=2, G=4, seed=35)
    bt.tables[1, :4] = bt.tables[0, :4]
    bt.tables[2, 1] = bt.tables[2, 0]
    d = bt.dev()
    args = (d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"])
    out, lse = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"])
    o, l, to, tl = ref.attention(bt)
    assert_within(out, o, to, "out")
    assert_within(lse, l, tl, "lse")
    m = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"])
    want, tol = ref.mass(bt, lse.cpu(), m.shape[2])
    assert_within(m, want, tol, "mass")


def results(nrc, bt, cache, tables):
    """Bits of every operator on bt's sequences in this cache."""
    d = bt.dev()
    args = (d["q"], cache, tables, d["ctx_lens"], d["q_starts"])
    out, lse = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"])
    m = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], width=400)
    p = torch.arange(400, **I32).expand(bt.B, bt.H, 400).contiguous().cuda()
    got = nrc.context_kv_evict(cache, tables, d["ctx_lens"], m, p, d["ctx_lens"], 100, 4, 16)
    return out, lse, m, *got


@pytest.mark.parametrize("nodes", [2, 40])
@pytest.mark.parametrize("far", ["blocks", "pages", "heads"])
def test_cells_past_32_bits(nrc, nodes, far):
    """The same bits wherever the cells lie: blocks, page rows or heads more than 2^32 elements apart from the first."""
    bt = ref.Batch([300, 130], [nodes, 3], H=2, G=4, seed=36)
    want = results(nrc, bt, (near := bt.cache.cuda()), bt.tables.cuda())
    if far == "blocks":
        count = (1 << 20) + 3 * bt.nb
        view = torch.empty(count, 2, 16, 128, dtype=torch.bfloat16, device="cuda")
        place = count - 1 - 2 * torch.arange(bt.nb)
    else:
        shape = (16, 1 << 21, 2, 128) if far == "pages" else (2, 1 << 21, 16, 128)
        pool = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        view = pool.permute(1, 2, 0, 3) if far == "pages" else pool.permute(1, 0, 2, 3)
        place = (1 << 21) - 1 - 2 * torch.arange(bt.nb)
    assert view.stride(0) * int(place[0]) + view.stride(1) + 15 * view.stride(2) > 1 << 32
    for i in range(bt.nb):
        view[int(place[i])] = bt.cache[i].cuda()
    tables = torch.where(bt.tables >= 0, place[bt.tables.clamp(min=0).long()], -1).int().cuda()
    got = results(nrc, bt, view, tables)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    moved = torch.stack([view[int(p)] for p in place])
    assert torch.equal(moved.view(torch.int16), near.view(torch.int16))


def test_calls_on_two_streams_at_once(nrc):
    bts = [ref.Batch([3000, 500], [nodes, 3], H=2, G=4, seed=37 + nodes) for nodes in (4, 40)]
    ds = [bt.dev() for bt in bts]

    def step(d, cache, stream=None):
        args = (d["q"], cache, d["tables"], d["ctx_lens"], d["q_starts"])
        out, lse = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"], stream=stream)
        m = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], stream=stream)
        return out, lse, m, *nrc.context_kv_evict(cache, d["tables"], d["ctx_lens"], m, pos[id(d)], d["ctx_lens"], 700,
                                                  stream=stream)

    pos = {}
    for d in ds:
        cells = d["tables"].shape[1] * 16
        pos[id(d)] = torch.arange(cells, **I32).expand(2, 2, cells).contiguous().cuda()
    want = [step(d, d["cache"].clone()) for d in ds]
    caches = [[d["cache"].clone() for d in ds] for _ in range(4)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [[step(d, c, s) for d, c, s in zip(ds, cs, streams)] for cs in caches]
    torch.cuda.synchronize()
    for turn in got:
        for g, w in zip(turn, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))
