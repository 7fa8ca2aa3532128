"""Edges of the operators on a drafted token's way to the cache, on the GPU."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from draft_ref import dense_attention, gains_grad, make_batch, sum_depth  # noqa: E402
from test_draft_edges_abi import gains_inputs  # noqa: E402
from test_gpu_qk_norm import dev, inputs, within  # noqa: E402

Batch = make_batch()


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


@pytest.mark.parametrize("missing", ["q", "k", "both"])
def test_gradients_that_count_as_zero_on_another_stream(nrc, missing):
    """The current stream busy, its free memory full of NaN: the call on a side stream waits for neither."""
    i = inputs(700, 8, 4, 64, 64, torch.bfloat16, torch.float32, 12)
    args = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    gq, gk = dev(i["gq"]), dev(i["gk"])
    given = [None if missing in ("q", "both") else gq, None if missing in ("k", "both") else gk]
    want = nrc.qk_norm_rotate_grad(*(torch.zeros_like(z) if g is None else g for g, z in zip(given, (gq, gk))), *args)
    a = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        trash = [torch.full_like(t, math.nan) for t in (gq, gk, gq, gk)]
        torch.cuda.synchronize()
        del trash
        for _ in range(10):
            b = a @ a
        got = nrc.qk_norm_rotate_grad(*given, *args, stream=side)
        later = [torch.full_like(t, math.nan) for t in (gq, gk)]
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        torch.cuda.synchronize()
        del later, b


def test_dual_tensors_are_refused(nrc):
    import torch.autograd.forward_ad as forward

    i = inputs(4, 2, 2, 64, 64, torch.float32, None, 3)
    q, k, pos, cs = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"])]
    want = nrc.qk_norm_rotate(q, k, pos, cs)
    with forward.dual_level():
        dual = forward.make_dual(q, torch.ones_like(q))
        for call in (lambda: nrc.rope_rotate(dual, pos, cs), lambda: nrc.qk_norm_rotate(dual, k, pos, cs)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
        got = nrc.qk_norm_rotate(forward.unpack_dual(dual).primal, k, pos, cs)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("q_gains", [False, True])
def test_keys_without_heads(nrc, q_gains):
    """The gradients are those without keys, and 0 of the gains of none; through autograd too."""
    i = inputs(5, 3, 2, 64, 64, torch.bfloat16, torch.float32, 4)
    q, k, pos, cs, qw, kw = [dev(t) for t in (i["q"], i["k"][:, :0], i["pos"], i["cs"], *i["w"])]
    qw = qw if q_gains else None
    gq = dev(i["gq"])
    want = nrc.qk_norm_rotate_grad(gq, None, q, None, pos, cs, qw)
    got = nrc.qk_norm_rotate_grad(gq, k, q, k, pos, cs, qw, kw)
    assert torch.equal(got[0], want[0]) and got[1].shape == k.shape and torch.equal(got[3], torch.zeros_like(kw))
    assert got[2] is None if qw is None else torch.equal(got[2], want[2])
    q.requires_grad_(), kw.requires_grad_()
    out, none = nrc.qk_norm_rotate(q, k, pos, cs, qw, kw)
    assert none.shape == k.shape
    grads = torch.autograd.grad(out, (q, kw), gq)
    assert torch.equal(grads[0], want[0]) and torch.equal(grads[1], torch.zeros_like(kw))


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["by heads", "heads first", "one head", "into the third part"])
def test_parts_of_one_tensor_by_turns(nrc, kind, dtype, T):
    """Queries, keys and values head by head in one tensor, in place or from part to part: the results are those of new outputs."""
    H, d = (1 if kind == "one head" else 5), 64
    gen = torch.Generator().manual_seed(T)
    if kind == "heads first":
        wide = torch.randn(H, T, 3, d, generator=gen).to(dtype).cuda().transpose(0, 1)
    else:
        wide = torch.randn(T, H, 3, d, generator=gen).to(dtype).cuda()
    q, k, v = wide.unbind(2)
    pos = torch.randint(0, 50, (T,), generator=gen).cuda()
    cs = nrc.rope_table(50, d, dtype=torch.float32)
    want = nrc.qk_norm_rotate(q.clone(), k.clone(), pos, cs)
    kept = [q.clone(), k.clone(), v.clone()]
    if kind == "into the third part":
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=v, out_k=k)
        assert torch.equal(v, want[0]) and torch.equal(k, want[1]) and torch.equal(q, kept[0])
    else:
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=q, out_k=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept[2])


@pytest.mark.parametrize("kind", ["side by side", "head by head", "layers inside"])
@pytest.mark.parametrize("L,T,H", [(3, 5, 4), (1, 7, 2), (2, 1, 1)])
def test_cells_loaded_into_one_tensor(nrc, L, T, H, kind):
    """K's and V's rows by turns, as a projection leaves them: what new outputs hold, and nothing else is written."""
    gen = torch.Generator().manual_seed(T)
    blocks, bs = T // 4 + 2, 4
    caches = torch.zeros(L, blocks, H, nrc.fp4_page_bytes(bs), dtype=torch.uint8, device="cuda")
    slots = torch.randperm(blocks * bs, generator=gen)[:T].cuda()
    rows = torch.randn(2, L, T, H, 64, generator=gen).bfloat16().cuda()
    nrc.context_fp4_store(rows[0], rows[1], slots, caches)
    want = nrc.context_fp4_load(caches, slots)
    if kind == "side by side":
        wide = torch.full((L, T, 3, H, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        k, v, rest = wide.unbind(2)
    elif kind == "head by head":
        wide = torch.full((L, T, H, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        k, v, rest = wide.unbind(3)
    else:
        wide = torch.full((T, H, L, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda").permute(2, 0, 1, 3, 4)
        k, v, rest = wide.unbind(3)
    got = nrc.context_fp4_load(caches, slots, k, v)
    assert got[0] is k and got[1] is v
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and bool((rest == 7).all())


def attend(nrc, bt, packed, **kw):
    d = bt.dev()
    args = (d["q"], d["cache"] if packed is None else packed, d["tables"], d["ctx_lens"], d["q_starts"], d["max_nodes"])
    if packed is None:
        return nrc.context_window_attention(*args, bt.window, bt.sinks, **kw)
    return nrc.context_fp4_attention(*args, window=bt.window or 0, sinks=bt.sinks, **kw)


def attention_within(got, want):
    out, lse, tol_o, tol_l = want
    empty = lse == -math.inf
    assert torch.equal(got[1] == -math.inf, empty) and bool((got[0][empty] == 0).all())
    bad = ~((got[0].double() - out).abs() <= tol_o + 1e-30)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4], got[0][bad][:4], out[bad][:4], tol_o[bad][:4])
    bad = ~(((got[1].double() - lse).abs() <= tol_l) | empty)
    assert not bool(bad.any()), (int(bad.sum()), bad.nonzero()[:4], got[1][bad][:4], lse[bad][:4])


@pytest.mark.parametrize("fp4,window", [(True, None), (True, 1100), (False, 1100)])
@pytest.mark.parametrize("nodes", [12, 30])  # workgroups of 4 waves and of 8
@pytest.mark.parametrize("bs", [16, 24, 64, 1])
@pytest.mark.parametrize("gone", ["first", "middle", "last", "several", "most"])
def test_missing_blocks_among_whole_tiles(nrc, gone, bs, nodes, fp4, window):
    """Blocks that are not there in tiles of 128 keys that every row would see whole: the tiles before them, theirs, those behind."""
    bt = Batch([1700, 1300], [nodes, nodes - 3], H=1, G=8, block_size=bs, tree=False, seed=bs + nodes).behind(window, 5)
    packed = bt.pack(nrc) if fp4 else None
    first, last = (640 // bs, 1600 // bs)  # (of the keys that all rows see)
    for at, byte in dict(first=[(first, -1)], middle=[(1000 // bs, bt.nb)], last=[(last, -2 ** 31)],
                         several=[(first + 1, -1), (1000 // bs, -1), (last, -1)],
                         most=[(i, -1) for i in range(first, last) if i % 7]).items():
        if at == gone:
            for i, page in byte:
                bt.tables[0, i] = page
    attention_within(attend(nrc, bt, packed), dense_attention(bt))


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("bs,gone", [(1, []), (1, [2900]), (1, [700, 1900]), (2, [1200])])
def test_shares_of_many_blocks(nrc, bs, gone, fp4):
    """A workgroup's keys in more than a thousand blocks, with some that are not there."""
    nodes = [256, 250, 200, 256]
    bt = Batch([3100, 3000, 2500, 3199], nodes, H=8, G=8, block_size=bs, tree=False, seed=bs).behind(3000, 5)
    need = nrc._load().nrc_context_window_attention_workspace_bytes(4, sum(nodes), 64, 8, 256, 3199, 3000, 5)
    assert need == 0  # not split: a workgroup's share is all that its rows see
    packed = bt.pack(nrc) if fp4 else None
    for i in gone:
        bt.tables[1:, i // bs] = -1
    attention_within(attend(nrc, bt, packed, max_ctx=3199), dense_attention(bt))


def test_pages_of_other_sizes_give_the_same_bits(nrc):
    """A long share's tiles go the same way whatever the pages: the same keys in 263, 1050 and 4200 blocks."""
    ctx, n, H = 16500, 300, 32
    bt = Batch([ctx], [n], H=H, G=8, block_size=64, tree=False, seed=4, spare=0).behind(17000)
    assert nrc._load().nrc_context_window_attention_workspace_bytes(1, n, 8 * H, H, n, ctx, 17000, 0) == 0  # not split
    keys = bt.cache[bt.tables[0].long()].transpose(1, 2).flatten(0, 1)  # in their order
    want = None
    for bs in (64, 16, 4):
        bt.bs, bt.nb = bs, keys.shape[0] // bs
        order = torch.randperm(bt.nb, generator=torch.Generator().manual_seed(bs))
        bt.cache = torch.empty(bt.nb, H, bs, 128, dtype=torch.bfloat16)
        bt.cache[order] = keys.unflatten(0, (bt.nb, bs)).transpose(1, 2)
        bt.tables = order.to(torch.int32)[None]
        packed = bt.pack(nrc)
        got = attend(nrc, bt, packed, max_ctx=ctx)
        if want is None:
            want = got
            attention_within(got, dense_attention(bt))
        assert all(torch.equal(a, b) for a, b in zip(got, want)), bs


@pytest.mark.parametrize("along", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d", [(4099, 23, 3, 64), (20000, 5, 1, 64), (3001, 2, 31, 128), (70000, 8, 2, 64)])
def test_gains_gradients_of_many_rows(nrc, T, Hq, Hk, d, along):
    """By the depth of the sums: one row that is lost or counted twice is outside the bound."""
    parts = [gains_inputs(T, h, d, along, T + h) for h in (Hq, Hk)]
    pos, cs = parts[0][3], parts[0][4]
    if along:  # (the keys' gradients are along the outputs of their own positions)
        parts[1] = (*parts[1][:3], pos, cs)
        from draft_ref import turn

        parts[1] = (parts[1][0], turn(parts[1][0].double(), pos, cs, "half")[0].bfloat16(), *parts[1][2:])
    (q, gq, qw, *_), (k, gk, kw, *_) = parts
    back = nrc.qk_norm_rotate_grad(*(dev(t) for t in (gq, gk, q, k, pos, cs, qw, kw)), layout="half")
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for i, (x, g, w, h, o) in enumerate(((q, gq, qw, Hq, Hk), (k, gk, kw, Hk, Hq))):
        within(back[2 + i], *gains_grad(g, x, w, pos, cs, "half", 1e-6, sum_depth(T, h, o, d // 16, cus)))


@pytest.mark.parametrize("wanted", ["q", "k", "qw", "kw", "q kw", "q qw", "k kw", "q k qw kw"])
def test_frozen_parts_are_not_worked_out(nrc, monkeypatch, wanted):
    """Gradients of some inputs: those of all, without the queries' or the keys' work where nobody asks for it."""
    i = inputs(30, 4, 2, 64, 32, torch.bfloat16, torch.float32, 6)
    all_of = dict(zip(("q", "k", "pos", "cs", "qw", "kw"), (dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"]))))
    gq, gk = dev(i["gq"]), dev(i["gk"])
    full = dict(zip(("q", "k", "qw", "kw"), nrc.qk_norm_rotate_grad(gq, gk, *all_of.values())))
    names = wanted.split()
    leaves = [all_of[n].requires_grad_() for n in names]
    heads, plain = [], nrc.qk_norm_rotate_grad

    def counted(grad_q, grad_k, q, k, *rest, **kw):
        heads.append(q.shape[1] + (0 if k is None else k.shape[1]))
        return plain(grad_q, grad_k, q, k, *rest, **kw)

    monkeypatch.setattr(nrc, "qk_norm_rotate_grad", counted)
    out = nrc.qk_norm_rotate(*all_of.values())
    got = torch.autograd.grad(out, leaves, (gq, gk))
    assert heads == [4 * any(n[0] == "q" for n in names) + 2 * any(n[0] == "k" for n in names)]
    tols = {n + "w": gains_grad(i["g" + n], i[n], w, i["pos"], i["cs"], "interleaved", 1e-6, sum_depth(30, h, 6 - h, 4, 256))[1]
            for n, w, h in zip("qk", i["w"], (4, 2))}
    for n, g in zip(names, got):
        # (another number of workgroups: the gains' sums in another order, each within the bound)
        assert torch.equal(g, full[n]) if n in "qk" else bool(((g - full[n]).abs().cpu() <= 2 * tols[n]).all())
