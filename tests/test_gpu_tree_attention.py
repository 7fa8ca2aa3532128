"""context_tree_attention and context_attention_mass against 64-bit references."""

import math

import numpy as np
import pytest

import cache_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def run(nrc, bt, **kw):
    d = bt.dev()
    args = (d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"])
    out, lse = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"], **kw)
    torch.cuda.synchronize()
    return out, lse, args, d


def assert_within(got, want, tol, what):
    got = got.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    same = (got == want) | torch.isnan(want)
    off = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(off <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, the worst by {float((off - tol).max())}"


def check(nrc, bt, cap=0.0, scale=None, mass=True, **kw):
    kw = dict(kw, softcap=cap, **({} if scale is None else {"scale": scale}))
    out, lse, args, d = run(nrc, bt, **kw)
    sc = 0.125 if scale is None else scale
    o, l, to, tl = ref.attention(bt, sc, cap)
    assert_within(out, o, to, "out")
    assert_within(lse, l, tl, "lse")
    if mass:
        width = max(c + n for c, n in zip(bt.ctx, bt.nodes)) + 5
        l32 = l.float()
        gen = torch.Generator().manual_seed(9)
        w = torch.rand(bt.B, bt.H, width, generator=gen)
        got = nrc.context_attention_mass(*args, l32.cuda(), d["max_nodes"], tree_mask=d["tree_mask"], weights=w.cuda(),
                                         decay=0.75, **kw)
        want, tol = ref.mass(bt, l32, width, w, 0.75, sc, cap)
        assert_within(got, want, tol, "mass")
    return out, lse


# contexts from nothing over whole and broken tiles and pages, one node and several
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 31, 32, 33, 64, 100, 257])
@pytest.mark.parametrize("nodes", [1, 7])
def test_lengths(nrc, ctx, nodes):
    check(nrc, ref.Batch([ctx], [nodes], seed=ctx + nodes))


@pytest.mark.parametrize("block_size", [1, 3, 8, 16, 24, 32, 48, 128])
def test_block_sizes(nrc, block_size):
    check(nrc, ref.Batch([70, 5, 131], [9, 1, 4], block_size=block_size, seed=block_size))


# query rows per KV head from one to several blocks of them, every tile count
@pytest.mark.parametrize("H,G,nodes", [(1, 1, 1), (8, 1, 2), (2, 3, 5), (1, 16, 1), (1, 8, 3), (4, 5, 5), (1, 7, 9),
                                       (1, 8, 9), (2, 4, 33), (1, 2, 70)])
def test_heads_and_rows(nrc, H, G, nodes):
    check(nrc, ref.Batch([50, 77], [nodes, max(1, nodes - 2)], H=H, G=G, seed=H + 10 * G))


@pytest.mark.parametrize("nodes", [1, 2, 31, 32, 33, 65])
def test_chain(nrc, nodes):
    check(nrc, ref.Batch([40, 0], [nodes, nodes], tree=False, seed=nodes))


@pytest.mark.parametrize("cap", [1.0, 30.0])
def test_softcap(nrc, cap):
    check(nrc, ref.Batch([90, 33], [6, 40], seed=3, q_scale=6.0), cap=cap)


def test_scale(nrc):
    check(nrc, ref.Batch([90, 33], [6, 4], seed=4), scale=0.031)


@pytest.mark.parametrize("scale,cap", [(2.0 ** -40, 0.0), (2.0 ** 40, 0.0), (0.125, 2.0 ** -10), (0.125, 2.0 ** 10),
                                       (2.0 ** -40, 2.0 ** 10), (2.0 ** 40, 2.0 ** -10), (2.0 ** 40, 2.0 ** 10)])
@pytest.mark.parametrize("nodes", [5, 40])
def test_ends_of_the_scales(nrc, scale, cap, nodes):
    # (scores of 2^40 and FP32's lse of them are 2^17 apart at the nearest, or equal: no weight to compare)
    check(nrc, ref.Batch([90, 33], [nodes, 6], seed=38), scale=scale, cap=cap, mass=cap > 0 or scale < 1)


@pytest.mark.parametrize("size", [1e3, 1e6, 1e10, 1e15])
@pytest.mark.parametrize("nodes", [5, 40])
def test_scores_whose_spacing_passes_the_exponent(nrc, size, nodes):
    """Scores of up to 1e30, where FP32's neighbours differ by more than an exponential holds: one key takes a row, or
    equal ones share it; the sums are exact (one element of q and k each), so the same key as in 64 bits."""
    bt = ref.Batch([90, 33], [nodes, 6], seed=39, tree=False)
    q, k = bt.q[..., :1].clone(), bt.cache[..., :1].clone()
    bt.q.zero_()
    bt.cache[..., :64] = 0
    bt.q[..., :1], bt.cache[..., :1] = q * size, k * size
    out, lse, args, d = run(nrc, bt)
    o, l, _, _ = ref.attention(bt)
    big = (l.abs() > 2.0 ** 32)[..., None]
    # beyond 2^32 the next score is e^-250 away at least: out is V itself, or the mean of equal keys' V (bf16 weights
    # that are all 1, an FP32 sum, a reciprocal and the product with it, one rounding)
    off = torch.where(big, (out.double().cpu() - o).abs() - o.abs() * 2.0 ** -8 - 2.0 ** -18 * 6, -1.0)
    assert bool((off <= 0).all()) and bool(torch.isfinite(out).all())
    # lse: base (two roundings), its factors (three) and 24 of log2's own steps
    assert bool(((lse.double().cpu() - l).abs() <= l.abs() * 6 * 2.0 ** -24 + 1e-3 + 64 * 2.0 ** -23 * l.abs()).all())
    m = nrc.context_attention_mass(*args, lse, d["max_nodes"])
    assert bool((m >= 0).all())


def test_ragged_batch_with_empty_sequences(nrc):
    check(nrc, ref.Batch([0, 40, 7, 0, 200], [0, 3, 0, 5, 1], seed=5))


def test_long_contexts_are_split(nrc):
    """One sequence, few heads: the context is split over workgroups and joined."""
    bt = ref.Batch([5000, 1300, 3], [3, 2, 1], H=1, G=2, seed=6)
    assert nrc._load().nrc_context_tree_attention_workspace_bytes(bt.B, bt.T, 2, 1, 3, 5000) > 0
    check(nrc, bt, max_ctx=5000)
    check(nrc, bt, cap=20.0, max_ctx=5000)


@pytest.mark.parametrize("ctx,nodes,H,G", [([3000, 0, 900, 130], [30, 20, 0, 33], 1, 4), ([1500, 700], [40, 33], 2, 8),
                                           ([2100, 64, 128], [100, 3, 70], 1, 6), ([1000] * 70, [9] * 70, 1, 8)])
def test_large_trees_over_split_contexts(nrc, ctx, nodes, H, G):
    """Many rows: shares by the lengths, empty sequences, several row blocks, more sequences than a wave's lanes."""
    bt = ref.Batch(ctx, nodes, H=H, G=G, seed=sum(ctx))
    need = nrc._load().nrc_context_tree_attention_workspace_bytes(bt.B, bt.T, H * G, H, bt.max_nodes, max(ctx))
    assert need > 0
    check(nrc, bt, max_ctx=max(ctx))
    check(nrc, ref.Batch(ctx, nodes, H=H, G=G, seed=1, tree=False), cap=25.0, max_ctx=max(ctx), mass=False)


def test_large_trees_with_absent_blocks_and_odd_values(nrc):
    """Tiles with keys that are not there among whole ones; NaN and infinities in a node of a large tree."""
    bt = ref.Batch([1000, 600], [40, 40], H=1, G=4, seed=30)
    bt.tables[0, 20] = -1
    bt.tables[0, 21] = bt.nb
    bt.tables[1, 3] = 2 ** 31 - 1
    check(nrc, bt)
    for bad in (math.nan, math.inf, -math.inf):
        b2 = ref.Batch([1000, 600], [40, 40], H=1, G=4, seed=31)
        o, l, to, tl = ref.attention(b2)
        c = b2.cell(1, 600 + 5)
        b2.cache[c[0], :, c[1], 64 + 9] = bad
        out, lse, args, d = run(nrc, b2)
        sees = torch.from_numpy(np.array([i >= 40 and ref.bits(b2.mask[i], 40)[5] for i in range(80)]))
        assert_within(out[~sees.cuda()], o[~sees], to[~sees], "out")
        hit = out[sees.cuda()].float().cpu()
        assert bool((torch.isnan(hit[..., 9]) if math.isnan(bad) else hit[..., 9] == bad).all())
        rest = [i for i in range(64) if i != 9]
        assert_within(out[sees.cuda()][..., rest], o[sees][..., rest], to[sees][..., rest], "out beside it")
        assert_within(lse, l, tl, "lse")


def test_large_scores_and_equal_scores(nrc):
    """Scores that rise along the context (the running maximum moves), and scores all equal."""
    bt = ref.Batch([300], [2], H=1, G=2, seed=7, q_scale=1.0)
    for j in range(302):
        c = bt.cell(0, j)
        bt.cache[c[0], :, c[1], :64] = (j - 150) / 16.0
    bt.q[:] = 1.0
    check(nrc, bt)
    bt.q[:] = 0.0
    check(nrc, bt)
    bt.q[:] = -1.0
    check(nrc, bt)


def test_rows_that_see_nothing(nrc):
    """No context and an empty mask: 0 and -inf; and they add no weight."""
    bt = ref.Batch([0, 0, 20], [5, 40, 3], seed=8)
    bt.mask[1] = 0
    bt.mask[5 + 33] = 0
    bt.mask[45] = 0
    out, lse = check(nrc, bt)
    assert bool((out[1] == 0).all()) and bool((lse[1] == -math.inf).all()) and bool((lse[38] == -math.inf).all())


def test_any_mask(nrc):
    """Masks that are no trees: later nodes seen, itself not, bits past the nodes set."""
    bt = ref.Batch([10, 33], [50, 35], seed=10)
    gen = torch.Generator().manual_seed(1)
    bt.mask = torch.randint(-2 ** 62, 2 ** 62, bt.mask.shape, generator=gen)
    check(nrc, bt)
    bt = ref.Batch([10, 33], [100, 70], G=1, seed=11, words=3)
    bt.mask = torch.randint(-2 ** 62, 2 ** 62, bt.mask.shape, generator=gen)
    check(nrc, bt)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_infinities_and_nan_in_unseen_keys(nrc, bad):
    """A node's K and V that only it and its descendants see reach no other row."""
    bt = ref.Batch([37], [20], H=1, G=2, seed=12)
    at = 11
    for part in (slice(0, 64), slice(64, 128), slice(70, 71)):
        b2 = ref.Batch([37], [20], H=1, G=2, seed=12)
        c = b2.cell(0, 37 + at)
        b2.cache[c[0], :, c[1], part] = bad
        out, lse, args, d = run(nrc, b2)
        o, l, to, tl = ref.attention(bt)
        sees = np.array([ref.bits(bt.mask[i], 20)[at] for i in range(20)])
        keep = torch.from_numpy(~sees)
        assert_within(out[keep.cuda()], o[keep], to[keep], "out")
        assert_within(lse[keep.cuda()], l[keep], tl[keep], "lse")
        hit = out[torch.from_numpy(sees).cuda()].float()
        if part.start >= 64:
            if math.isnan(bad):
                assert bool(torch.isnan(hit[..., part.start - 64:part.stop - 64]).all())
            else:
                assert bool((hit[..., part.start - 64:part.stop - 64] == bad).all())
            if part.stop == 71:
                rest = torch.cat([hit[..., :6], hit[..., 7:]], -1)
                assert bool(torch.isfinite(rest).all())
        elif math.isnan(bad):
            assert bool(torch.isnan(hit).all())


def test_nan_after_the_last_key(nrc):
    """What lies behind a sequence in its last page, and in blocks of no sequence, is not looked at."""
    bt = ref.Batch([37, 3], [2, 1], H=2, G=2, seed=13)
    used = {bt.cell(b, j) for b in range(2) for j in range(bt.ctx[b] + bt.nodes[b])}
    for p in range(bt.nb):
        for s in range(bt.bs):
            if (p, s) not in used:
                bt.cache[p, :, s] = math.nan
    check(nrc, bt)


def test_absent_blocks(nrc):
    """Keys whose block is no block are seen by nobody."""
    bt = ref.Batch([200, 40], [20, 5], seed=14)
    bt.tables[0, 2] = -1
    bt.tables[0, 5] = bt.nb
    bt.tables[0, 13] = 2 ** 31 - 1
    check(nrc, bt)
    bt.tables[:] = -1
    out, lse = check(nrc, bt)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_strided_views(nrc):
    """q as a column range of a wider row, a cache of other strides, tables of a wider array."""
    bt = ref.Batch([70, 20], [5, 3], seed=15)
    d = bt.dev()
    T, Hq, _ = bt.q.shape
    wide = torch.zeros(T, Hq + 3, 72, dtype=torch.bfloat16, device="cuda")
    q = wide[:, 1:1 + Hq, 8:72]
    q.copy_(d["q"])
    pool = torch.full((bt.nb, bt.bs, bt.H + 1, 136), math.nan, dtype=torch.bfloat16, device="cuda")
    cache = pool.permute(0, 2, 1, 3)[:, 1:, :, :128]
    cache.copy_(d["cache"])
    tables = torch.full((2, bt.tables.shape[1] + 5), 99, dtype=torch.int32, device="cuda")
    tables[:, :bt.tables.shape[1]] = d["tables"]
    out, lse = nrc.context_tree_attention(q, cache, tables[:, :bt.tables.shape[1]], d["ctx_lens"], d["q_starts"],
                                          bt.max_nodes, tree_mask=d["tree_mask"])
    want_o, want_l = nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"],
                                                bt.max_nodes, tree_mask=d["tree_mask"])
    assert torch.equal(out, want_o) and torch.equal(lse, want_l)
    width = 80
    got = torch.full((bt.H, 2, width + 3), -3.0, device="cuda").permute(1, 0, 2)[:, :, 1:1 + width]
    nrc.context_attention_mass(q, cache, tables[:, :bt.tables.shape[1]], d["ctx_lens"], d["q_starts"], lse,
                               bt.max_nodes, tree_mask=d["tree_mask"], out=got)
    plain = nrc.context_attention_mass(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], lse,
                                       bt.max_nodes, tree_mask=d["tree_mask"], width=width)
    assert torch.equal(got, plain)


def test_rows_of_no_sequence_stay(nrc):
    """Rows before the first and behind the last sequence, and past max_nodes, are left as they were."""
    bt = ref.Batch([20, 30], [3, 6], seed=16)
    d = bt.dev()
    q = torch.cat([d["q"][:2], d["q"], d["q"][:3]])
    mask = torch.cat([d["tree_mask"][:2], d["tree_mask"], d["tree_mask"][:3]])
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 6.0, device="cuda")
    nrc.context_tree_attention(q, d["cache"], d["tables"], d["ctx_lens"], d["q_starts"] + 2, 6, tree_mask=mask, out=out,
                               lse=lse)
    want, wl = nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], 6,
                                          tree_mask=d["tree_mask"])
    assert torch.equal(out[2:11], want) and torch.equal(lse[2:11], wl)
    assert bool((out[:2] == 5).all()) and bool((out[11:] == 5).all()) and bool((lse[11:] == 6).all())
    out.fill_(5.0)
    nrc.context_tree_attention(q, d["cache"], d["tables"], d["ctx_lens"], d["q_starts"] + 2, 4, tree_mask=mask, out=out)
    assert torch.equal(out[2:5], want[:3]) and bool((out[9:11] == 5).all())


def test_sizes_that_do_not_fit(nrc):
    """Row ranges outside q write nothing; a negative context counts as none; a longer one is cut."""
    bt = ref.Batch([20, 30], [3, 6], seed=17)
    d = bt.dev()
    out = torch.full(d["q"].shape, 5.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 3, 99], [-2, 3, 3], [5, 3, 3]):
        s = torch.tensor(starts, dtype=torch.int32, device="cuda")
        nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], s, 6, tree_mask=d["tree_mask"], out=out)
        assert bool((out[3:] == 5).all())
    cut = ref.Batch([20, 30], [3, 6], seed=17)
    cut.ctx = [0, 12]
    lens = torch.tensor([-4, 30], dtype=torch.int32, device="cuda")
    got, _ = nrc.context_tree_attention(d["q"], d["cache"], d["tables"], lens, d["q_starts"], 6,
                                        tree_mask=d["tree_mask"], max_ctx=12)
    o, l, to, tl = ref.attention(cut)
    assert_within(got, o, to, "out")


def test_deterministic_and_on_its_stream(nrc):
    bt = ref.Batch([3000, 700], [9, 4], H=2, G=4, seed=18)
    out, lse, args, d = run(nrc, bt)
    for _ in range(3):
        o2, l2 = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"])
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3, l3 = nrc.context_tree_attention(*args, d["max_nodes"], tree_mask=d["tree_mask"], stream=s)
    m3 = nrc.context_attention_mass(*args, l3, d["max_nodes"], tree_mask=d["tree_mask"], stream=s)
    s.synchronize()
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    assert torch.equal(m3, nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"]))


def test_two_graphs_replayed_in_turn(nrc):
    """Two captured calls with workspaces of their own, replayed with eager work between."""
    bts = [ref.Batch([3000, 700], [9, 4], H=2, G=4, seed=s) for s in (19, 20)]
    ds = [bt.dev() for bt in bts]
    call = lambda d: nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"],
                                                d["max_nodes"], max_ctx=3000, tree_mask=d["tree_mask"])
    mass = lambda d, l: nrc.context_attention_mass(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], l,
                                                   d["max_nodes"], tree_mask=d["tree_mask"])
    eager = [call(d) for d in ds]
    masses = [mass(d, e[1]) for d, e in zip(ds, eager)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = call(d)
            outs.append((*o, mass(d, o[1])))
        graphs.append(g)
    for k in range(4):
        for g, o in zip(graphs, outs):
            for t in o:
                t.fill_(7.0)
            g.replay()
            call(ds[k % 2])
        torch.cuda.synchronize()
        for o, e, m in zip(outs, eager, masses):
            assert torch.equal(o[0], e[0]) and torch.equal(o[1], e[1]) and torch.equal(o[2], m)


def test_mass_in_place_and_without_weights(nrc):
    bt = ref.Batch([70, 20], [5, 3], seed=21)
    out, lse, args, d = run(nrc, bt)
    plain = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], width=90)
    want, tol = ref.mass(bt, lse.cpu(), 90)
    assert_within(plain, want, tol, "mass")
    w = torch.rand(2, bt.H, 90, device="cuda")
    w[:, :, 80:] = math.nan  # stale cells past every sequence
    w0 = w.clone()
    got = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], weights=w, out=w, decay=0.5)
    assert got is w
    want, tol = ref.mass(bt, lse.cpu(), 90, torch.nan_to_num(w0.cpu()), 0.5)
    assert_within(got, want, tol, "mass")
    assert bool((got[1, :, 23:] == 0).all())
    # a narrower width takes the first cells
    few = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], width=31)
    assert torch.equal(few, plain[:, :, :31].contiguous())


def test_mass_adds_up_to_the_rows(nrc):
    """Every row gives its keys one in all: N rows a head give N, within the summed roundings (2^-20 each key)."""
    bt = ref.Batch([1000, 64], [9, 64], H=2, G=2, seed=22)
    out, lse, args, d = run(nrc, bt)
    m = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"]).double().sum(-1).cpu()
    want = torch.tensor(bt.nodes, dtype=torch.float64)[:, None] * bt.G
    assert bool(((m - want).abs() <= want * 2.0 ** -14).all())


def test_refusals(nrc):
    bt = ref.Batch([70, 20], [5, 3], seed=23)
    d = bt.dev()
    ok = dict(q=d["q"], cache=d["cache"], tables=d["tables"], ctx_lens=d["ctx_lens"], q_starts=d["q_starts"], max_nodes=5,
              tree_mask=d["tree_mask"])
    nrc.context_tree_attention(**ok)
    bad = [dict(q=d["q"].float()), dict(q=d["q"].cpu()), dict(q=d["q"][:, :7]), dict(q=d["q"][..., :32]),
           dict(q=d["q"].transpose(1, 2)), dict(cache=d["cache"][..., :64]), dict(cache=d["cache"].half()),
           dict(tables=d["tables"].long()), dict(tables=d["tables"].cpu()), dict(tables=d["tables"][0]),
           dict(ctx_lens=d["ctx_lens"][:1]), dict(q_starts=d["q_starts"][:2]), dict(ctx_lens=d["ctx_lens"].long()),
           dict(max_nodes=0), dict(max_nodes=65), dict(max_nodes=2 ** 32 + 5), dict(max_nodes=70000),
           dict(tree_mask=d["tree_mask"][:3]), dict(tree_mask=d["tree_mask"].int()), dict(scale=0.0), dict(scale=-1.0),
           dict(scale=math.nan), dict(scale=1e-13), dict(softcap=-1.0), dict(softcap=math.inf), dict(softcap=2000.0),
           dict(max_ctx=2 ** 64 + 7), dict(max_ctx=-1), dict(max_ctx=2 ** 31),
           dict(out=torch.empty(8, 8, 64, device="cuda")), dict(lse=torch.empty(8, 7, device="cuda")),
           dict(stream=None, out=torch.empty(8, 8, 64, dtype=torch.bfloat16))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, nrc.NrcError)):
            nrc.context_tree_attention(**{**ok, **kw})
    lse = torch.zeros(8, 8, device="cuda")
    nrc.context_attention_mass(**ok, lse=lse)
    bad = [dict(lse=lse[:7]), dict(lse=lse.double()), dict(decay=math.nan), dict(weights=lse), dict(width=-1),
           dict(weights=torch.zeros(2, 2, 9, dtype=torch.float64, device="cuda")),
           dict(weights=torch.zeros(2, 2, 9, device="cuda"), width=8), dict(out=torch.zeros(2, 1, 9, device="cuda")),
           dict(out=torch.zeros(2, 1, 9, device="cuda").expand(2, 2, 9))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, RuntimeError, nrc.NrcError)):
            nrc.context_attention_mass(**{**ok, "lse": lse, **kw})


def test_empty_calls(nrc):
    bt = ref.Batch([70, 20], [5, 3], seed=24)
    d = bt.dev()
    q0 = d["q"][:0]
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = nrc.context_tree_attention(q0, d["cache"], d["tables"], d["ctx_lens"], z, 1)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    m = nrc.context_attention_mass(q0, d["cache"], d["tables"], d["ctx_lens"], z, lse, 1, weights=torch.ones(2, 2, 80, device="cuda"))
    assert bool((m[0, :, :70] == 1).all()) and bool((m[0, :, 70:] == 0).all()) and bool((m[1, :, 20:] == 0).all())
    out, lse = nrc.context_tree_attention(d["q"], d["cache"], d["tables"][:0], z[:0], z[:1], 1)
    torch.cuda.synchronize()
