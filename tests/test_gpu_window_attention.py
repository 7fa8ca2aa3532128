"""context_window_attention and context_fp4_attention against a 64-bit reference."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import cache_ref  # noqa: E402
from draft_ref import make_batch  # noqa: E402

Batch = make_batch()


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def run(nrc, bt, fp4, packed=None, **kw):
    d = bt.dev()
    cache, tables = d.pop("cache"), d.pop("tables")
    q, ctx, starts, nodes = d.pop("q"), d.pop("ctx_lens"), d.pop("q_starts"), d.pop("max_nodes")
    if fp4:
        return nrc.context_fp4_attention(q, packed, tables, ctx, starts, nodes, window=bt.window or 0, sinks=bt.sinks,
                                         **d, **kw)
    return nrc.context_window_attention(q, cache, tables, ctx, starts, nodes, bt.window, bt.sinks, **d, **kw)


def check(got, bt, cap=0.0, scale=0.125, rows=slice(None)):
    out, lse, tol_o, tol_l = (t[rows] for t in cache_ref.attention(bt, scale=scale, cap=cap))
    o, l = got[0].double().cpu()[rows], got[1].double().cpu()[rows]
    empty = lse == -math.inf
    assert torch.equal(l == -math.inf, empty)
    assert bool((o[empty] == 0).all())
    bad = ~((o - out).abs() <= tol_o + 1e-30)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4], o[bad][:4], out[bad][:4], tol_o[bad][:4])
    bad = ~(((l - lse).abs() <= tol_l) | empty)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4], l[bad][:4], lse[bad][:4])


# contexts, nodes, H, G, block_size, tree, window, sinks
SMALL = [
    ([0], [1], 1, 1, 16, False, 1, 0),
    ([5, 0, 40], [1, 1, 1], 2, 4, 16, False, 8, 2),
    ([1, 31, 32, 33, 64, 200], [1] * 6, 2, 8, 16, False, 32, 4),
    ([300, 17, 129], [5, 2, 1], 2, 3, 24, False, 50, 7),
    ([100, 7], [3, 4], 1, 5, 1, False, 33, 1),
    ([100, 64, 0], [5, 6, 7], 2, 4, 5, True, 20, 3),
    ([500, 77], [7, 1], 2, 4, 48, True, 100, 0),
    ([90, 200], [3, 30], 1, 1, 8, False, 4, 0),
    ([256, 130], [8, 8], 3, 2, 64, True, 1000, 500),
    ([70, 90], [16, 9], 2, 2, 16, False, 16, 40),  # sinks past some windows
    ([200, 3], [2, 0], 2, 4, 16, False, 1, 0),  # the row's own key alone
    ([33, 100], [5, 5], 1, 8, 32, True, 2, 1),  # a window below the trees' depths
]
MANY = [
    ([40, 0, 300], [40, 64, 33], 2, 4, 16, False, 50, 3),
    ([300, 9], [33, 20], 2, 5, 24, True, 64, 4),
    ([10], [333], 1, 3, 16, False, 100, 5),
    ([0], [520], 2, 1, 8, False, 32, 0),
    ([700, 100], [70, 9], 1, 8, 5, True, 129, 130),
    ([129], [140], 1, 8, 64, False, 1, 0),
    ([400], [65], 2, 1, 16, True, 4000, 0),
]


def batch(ctx, nodes, H, G, bs, tree, window, sinks, seed=1, **kw):
    return Batch(ctx, nodes, H=H, G=G, block_size=bs, tree=tree, seed=seed, **kw).behind(window, sinks)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("shape", SMALL + MANY)
def test_window(nrc, shape, cap, fp4):
    bt = batch(*shape)
    packed = bt.pack(nrc) if fp4 else None
    check(run(nrc, bt, fp4, packed, softcap=cap), bt, cap)


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("shape", SMALL + MANY)
def test_fp4_without_a_window(nrc, shape, cap):
    bt = batch(*shape)
    bt.window, bt.sinks = None, 9
    packed = bt.pack(nrc)
    check(run(nrc, bt, True, packed, softcap=cap), bt, cap)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("ctx,nodes,G,window", [([9000], [2], 4, 6000), ([9000, 100], [3, 3], 8, 5000), ([5000, 4000], [20, 3], 4, 3900),
                                                ([5000], [40], 8, 4000), ([4100], [1], 1, 2048)])
def test_long_windows_are_split(nrc, ctx, nodes, G, window, fp4):
    """Shares over workgroups, joined by a second launch."""
    bt = batch(ctx, nodes, 1, G, 16, False, window, 5)
    rows = nrc._load().nrc_context_window_attention_workspace_bytes(len(ctx), sum(nodes), G, 1, max(nodes), max(ctx), window, 5)
    assert rows > 0 or G == 1
    packed = bt.pack(nrc) if fp4 else None
    check(run(nrc, bt, fp4, packed), bt)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("nodes", [[3, 4], [50, 20]])
@pytest.mark.parametrize("bs", [16, 24])
def test_pages_that_are_not_there(nrc, bs, nodes, fp4):
    """Blocks outside the pool and keys past the table are seen by nobody, and rows left with none get 0 and -inf."""
    bt = batch([300, 200], nodes, 2, 4, bs, False, 60, 20, seed=3)
    packed = bt.pack(nrc) if fp4 else None
    bt.tables[0, 0] = -1
    bt.tables[0, (300 // bs) - 1] = bt.nb
    bt.tables[0, (300 // bs) - 2] = -2 ** 31
    bt.tables[1, :] = -1  # nothing at all
    check(run(nrc, bt, fp4, packed), bt)
    bt.tables = bt.tables[:, :300 // bs].contiguous()  # the last keys lie past the table
    check(run(nrc, bt, fp4, packed, max_ctx=300), bt)


@pytest.mark.parametrize("nodes,G", [([3], 4), ([40], 4)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_row_does_not_see_does_not_reach_it(nrc, nodes, G, bad):
    """K and V of bf16 keys before the windows, within the same tiles, and of nodes behind a row's own. (Rows of one wave move
    their references together, so others' NaN may move a row's roundings: the bound is the clean reference's.)"""
    for tree in (False, True):
        bt = batch([100], nodes, 2, G, 16, tree, 37, 2, seed=5)
        clean = bt.cache.clone()
        last = 100 + nodes[0] - 1
        for key in (3, 50, 62, 63, last if not tree else 20):
            c = bt.cell(0, key)
            bt.cache[c[0], :, c[1]] = bad
        got = run(nrc, bt, False)
        there = bt.sees(0, torch.ones(100 + nodes[0], dtype=torch.bool).numpy())
        hit = torch.zeros(nodes[0], dtype=torch.bool)
        for key in (3, 50, 62, 63, last if not tree else 20):
            hit |= there[:, key]
        assert not bool(hit.all())
        bt.cache = clean
        check(got, bt, rows=~hit)


def test_infinities_that_rows_see_reach_them(nrc):
    """V alone: an infinity seen with some weight gives an infinity, both signs or a NaN give NaN, in its element."""
    for nodes in ([3], [40]):
        bt = batch([64], nodes, 1, 4, 16, False, 10, 0, seed=6)
        c = bt.cell(0, 60)
        bt.cache[c[0], 0, c[1], 64 + 5] = math.inf
        bt.cache[c[0], 0, c[1], 64 + 6] = -math.inf
        bt.cache[c[0], 0, c[1], 64 + 7] = math.nan
        out, lse = run(nrc, bt, False)
        sees = torch.tensor([60 > 64 + i - 10 for i in range(nodes[0])]).cuda()
        assert bool((out[sees][..., 5] == math.inf).all()) and bool((out[sees][..., 6] == -math.inf).all())
        assert bool(out[sees][..., 7].isnan().all()) and bool(out[~sees].isfinite().all()) and bool(lse.isfinite().all())
        rest = [d for d in range(64) if d not in (5, 6, 7)]
        assert bool(out[..., rest].isfinite().all())


@pytest.mark.parametrize("nodes,G", [([3], 4), ([40], 4)])
def test_cells_of_4_bits_that_are_not_seen(nrc, nodes, G):
    """Any bytes in cells before the windows, behind a row's own node, behind the last node; NaN cells reach the rows that
    see them, out and lse."""
    gen = torch.Generator().manual_seed(2)
    for byte in (0xFF, 0xFE, 0x00, None):
        bt = batch([100], nodes, 2, G, 16, False, 37, 2, seed=5, spare=5)
        packed = bt.pack(nrc)
        clean = run(nrc, bt, True, packed)
        for key in [3, 50, 62] + list(range(100 + nodes[0], bt.tables.shape[1] * 16)):
            if bt.cell(0, key):
                bt.wipe(packed, 0, key, byte, gen)
        got = run(nrc, bt, True, packed)
        for a, b in zip(got, clean):
            assert torch.equal(a, b)
    bt.wipe(packed, 0, 63, 0xFF)  # seen by node 0 alone: 100 - 37 + 1 = 64 is the first key of its window
    got = run(nrc, bt, True, packed)
    assert all(torch.equal(a, b) for a, b in zip(got, clean))
    bt.wipe(packed, 0, 70, 0xFF)  # seen by nodes up to 6
    got = run(nrc, bt, True, packed)
    hit = torch.arange(nodes[0]) <= 6
    assert bool(got[0][hit.cuda()].isnan().all()) and bool(got[1][hit.cuda()].isnan().all())
    check(got, bt, rows=~hit)


def test_masks_that_leave_a_row_empty(nrc):
    for fp4 in (False, True):
        for nodes in ([4, 3], [40, 20]):
            bt = batch([0, 50], nodes, 2, 4, 16, True, 8, 0, seed=7)
            bt.mask[1] = 0  # no context: sees nothing
            bt.mask[nodes[0] + 1] = 0  # stands before its sequence's first node
            packed = bt.pack(nrc) if fp4 else None
            got = run(nrc, bt, fp4, packed)
            check(got, bt)
            assert bool((got[0][1] == 0).all()) and bool((got[1][1] == -math.inf).all())


def test_equal_to_the_attention_without(nrc):
    """A window that holds everything: the bound of the one applies to the other; bits of a mask past the nodes mean nothing."""
    bt = batch([130, 60], [20, 7], 2, 4, 16, True, 2 ** 31 - 1, 2 ** 31 - 1, seed=8, words=2)
    bt.mask[0] |= 1 << 40
    d = bt.dev()
    plain = nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], d["max_nodes"],
                                       tree_mask=d["tree_mask"])
    got = run(nrc, bt, False)
    assert bool(((got[0].float() - plain[0].float()).abs() <= 2.0 ** -6).all())
    check(got, bt)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("nodes", [[3, 2], [30, 44]])
def test_rows_of_no_sequence_and_given_outputs(nrc, nodes, fp4):
    bt = batch([60, 70], nodes, 2, 4, 16, False, 20, 4, seed=9)
    packed = bt.pack(nrc) if fp4 else None
    full = run(nrc, bt, fp4, packed)
    T = sum(nodes)
    wide = torch.randn(T + 5, 8, 64).bfloat16()
    wide[2:2 + T] = bt.q
    bt.q, bt.T, bt.q_starts = wide, T + 5, bt.q_starts + 2
    out, lse = run(nrc, bt, fp4, packed)
    inside = slice(2, 2 + T)
    assert torch.equal(out[inside], full[0]) and torch.equal(lse[inside], full[1])
    for rest in (out[:2], out[2 + T:]):
        assert bool((rest == 0).all())
    assert bool((lse[:2] == -math.inf).all()) and bool((lse[2 + T:] == -math.inf).all())
    mine, mine_lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    run(nrc, bt, fp4, packed, out=mine, lse=mine_lse)
    assert torch.equal(mine[inside], full[0]) and bool((mine[:2] == 7).all()) and bool((mine[2 + T:] == 7).all())
    assert bool((mine_lse[:2] == 7).all()) and torch.equal(mine_lse[inside], full[1])
    # rows past max_nodes
    bt.max_nodes = min(nodes)
    cut, _ = run(nrc, bt, fp4, packed)
    big = 0 if nodes[0] > nodes[1] else 1
    start = 2 + (0 if big == 0 else nodes[0])
    assert bool((cut[start + bt.max_nodes:start + max(nodes)] == 0).all())
    assert torch.equal(cut[start:start + bt.max_nodes], full[0][start - 2:start - 2 + bt.max_nodes])


@pytest.mark.parametrize("fp4", [False, True])
def test_no_sequences(nrc, fp4):
    bt = batch([10], [2], 2, 4, 16, False, 4, 0)
    packed = bt.pack(nrc) if fp4 else None
    bt.tables, bt.ctx_lens, bt.q_starts = bt.tables[:0], bt.ctx_lens[:0], bt.q_starts[:1]
    out, lse = run(nrc, bt, fp4, packed)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    bt.q = bt.q[:0]
    out, lse = run(nrc, bt, fp4, packed)
    assert out.shape == (0, 8, 64)


@pytest.mark.parametrize("fp4", [False, True])
def test_large_scores(nrc, fp4):
    """Scores of thousands, rows whose largest is far above the rest and comes last or first."""
    for nodes in ([2], [40]):
        bt = batch([200], nodes, 1, 4, 16, False, 150, 8, seed=11, q_scale=400.0)
        packed = bt.pack(nrc) if fp4 else None
        check(run(nrc, bt, fp4, packed), bt)
        check(run(nrc, bt, fp4, packed, softcap=50.0), bt, cap=50.0)
        check(run(nrc, bt, fp4, packed, scale=0.01), bt, scale=0.01)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("nodes", [[3, 2], [30, 44]])
def test_strides(nrc, nodes, fp4):
    """Queries inside wider rows, tables inside wider ones, pages with room between them."""
    bt = batch([60, 70], nodes, 2, 4, 16, False, 33, 4, seed=12)
    packed = bt.pack(nrc) if fp4 else None
    want = run(nrc, bt, fp4, packed)
    d = bt.dev()
    q = torch.zeros(bt.T, 11, 80, dtype=torch.bfloat16, device="cuda")[:, 2:10, 8:72]
    q.copy_(d["q"])
    tables = torch.zeros(2, 40, dtype=torch.int32, device="cuda")[:, 3:3 + bt.tables.shape[1]]
    tables.copy_(d["tables"])
    if fp4:
        page = packed.shape[2]
        cache = torch.zeros(2, bt.nb, page + 48, dtype=torch.uint8, device="cuda")[:, :, 16:16 + page].transpose(0, 1)
        cache.copy_(packed)
        got = nrc.context_fp4_attention(q, cache, tables, d["ctx_lens"], d["q_starts"], d["max_nodes"], window=33, sinks=4)
    else:
        cache = torch.zeros(2, bt.nb, 16, 144, dtype=torch.bfloat16, device="cuda")[..., 8:136].transpose(0, 1)
        cache.copy_(d["cache"])
        got = nrc.context_window_attention(q, cache, tables, d["ctx_lens"], d["q_starts"], d["max_nodes"], 33, 4)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("nodes,ctx", [([3], [5000]), ([60], [5000])])
def test_graph_streams_and_the_same_bits(nrc, nodes, ctx, fp4):
    bt = batch(ctx, nodes, 1, 4, 16, False, 4500, 4, seed=13)
    packed = bt.pack(nrc) if fp4 else None
    d = bt.dev()
    cache = packed if fp4 else d["cache"]
    f = nrc.context_fp4_attention if fp4 else nrc.context_window_attention
    call = lambda **kw: f(d["q"], cache, d["tables"], d["ctx_lens"], d["q_starts"], d["max_nodes"], window=4500, sinks=4,
                          max_ctx=5000, **kw)
    want = call()
    for a, b in zip(call(), want):
        assert torch.equal(a, b)
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        got.append(call(stream=s))
    for s, g in zip(sides, got):
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for _ in range(3):
        held[0].zero_(), held[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        call()


def test_refusals(nrc):
    bt = batch([60], [3], 2, 4, 16, False, 8, 2)
    packed = bt.pack(nrc)
    d = bt.dev()
    base = dict(q=d["q"], cache=d["cache"], tables=d["tables"], ctx_lens=d["ctx_lens"], q_starts=d["q_starts"], max_nodes=3,
                window=8, sinks=2)
    for bad in (dict(window=0), dict(window=-1), dict(window=2 ** 31), dict(window=1.5), dict(sinks=2 ** 31), dict(cache=packed),
                dict(q=d["q"].float()), dict(q=d["q"].cpu()), dict(tables=d["tables"].long()), dict(ctx_lens=d["ctx_lens"].long()),
                dict(out=torch.empty(3, 8, 64, device="cuda")), dict(lse=torch.empty(3, 8, device="cuda", dtype=torch.float64)),
                dict(max_ctx=-1), dict(tree_mask=torch.zeros(2, 1, dtype=torch.int64, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            nrc.context_window_attention(**{**base, **bad})
    for bad in (dict(sinks=-1), dict(max_nodes=0), dict(max_nodes=65536), dict(scale=0.0), dict(softcap=-1.0),
                dict(out=d["q"])):
        with pytest.raises(nrc.NrcError):
            nrc.context_window_attention(**{**base, **bad})
    base["cache"] = packed
    for bad in (dict(cache=d["cache"]), dict(cache=packed[..., :-16]), dict(cache=packed[0]), dict(cache=packed.cpu()),
                dict(window=2 ** 31), dict(tables=d["tables"].cpu())):
        with pytest.raises((TypeError, ValueError)):
            nrc.context_fp4_attention(**{**base, **bad})
    for bad in (dict(window=-1), dict(sinks=-1), dict(out=packed.view(torch.bfloat16).flatten()[:3 * 8 * 64].view(3, 8, 64)),
                dict(cache=torch.zeros(bt.nb, 2, 1104, dtype=torch.uint8, device="cuda")[..., 8:1096])):
        with pytest.raises(nrc.NrcError):
            nrc.context_fp4_attention(**{**base, **bad})
    for other in (nrc.context_tree_attention, nrc.context_attention_mass):
        with pytest.raises(TypeError, match="bfloat16"):
            kw = {k: v for k, v in base.items() if k not in ("window", "sinks")}
            other(**kw, **({} if other is nrc.context_tree_attention else dict(lse=torch.zeros(3, 8, device="cuda"))))
