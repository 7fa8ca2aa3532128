"""The operators around the cache at the edges of their calls: padded rows, outputs
made by the call."""

import math

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


def poison(*sizes):
    """Leaves memory of these sizes (bytes) in the allocator's hands that holds 0xA5."""
    torch.cuda.synchronize()
    held = [torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.synchronize()
    del held


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("H,d,R", [(2, 64, 64), (3, 96, 32), (1, 10, 6), (2, 66, 64)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate_padded_rows_come_out_as_they_went_in(nrc, dtype, layout, H, d, R, inverse):
    """Positions outside the table, in an output of the call's own: x's bits, NaN and infinities included."""
    T = 40
    gen = torch.Generator().manual_seed(d)
    x = torch.randn(T, H, d, generator=gen).to(dtype)
    x[3, 0, 1], x[3, 0, 2], x[5, 0, 0] = math.nan, math.inf, -0.0
    pos = torch.randint(0, 30, (T,), generator=gen)
    pos[::3], pos[5], pos[8], pos[39] = -1, 30, 2 ** 62, -2 ** 63
    x = x.cuda()
    table = nrc.rope_table(30, R)
    poison(x.numel() * x.element_size())
    out = nrc.rope_rotate(x, pos.cuda(), table, layout=layout, inverse=inverse)
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    outside = (pos < 0) | (pos >= 30)
    assert torch.equal(out.view(bits)[outside.cuda()], x.view(bits)[outside.cuda()])
    inside = nrc.rope_rotate(x[~outside.cuda()], pos[~outside].cuda(), table, layout=layout, inverse=inverse)
    assert torch.equal(out[~outside.cuda()], inside)


# few and many rows, each in one piece and split over workgroups
@pytest.mark.parametrize("ctx,nodes,H,G", [([20, 30], [3, 6], 2, 4), ([5000, 1300], [3, 2], 1, 2), ([900, 130], [30, 12], 1, 4),
                                           ([40, 33] * 40, [9, 12] * 40, 8, 4)])
def test_attention_rows_of_no_sequence(nrc, ctx, nodes, H, G):
    """Rows before the first sequence, behind the last and past max_nodes, in outputs of the call's own: 0 and -inf; the
    others' bits are those without such rows."""
    bt = ref.Batch(ctx, nodes, H=H, G=G, seed=50)
    d = bt.dev()
    before, behind = 5, 300
    q = torch.cat([d["q"][:1].expand(before, -1, -1), d["q"], d["q"][:1].expand(behind, -1, -1)])
    mask = torch.cat([d["tree_mask"][:1].expand(before, -1), d["tree_mask"], d["tree_mask"][:1].expand(behind, -1)])
    starts = d["q_starts"] + before
    T, Hq = q.shape[:2]
    want, want_l = nrc.context_tree_attention(d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], max(nodes),
                                              tree_mask=d["tree_mask"], max_ctx=max(ctx))
    for most in (max(nodes), min(nodes)):
        owned = torch.zeros(T, dtype=torch.bool)
        for b, n in enumerate(nodes):
            lo = before + int(bt.q_starts[b])
            owned[lo:lo + min(n, most)] = True
        owned = owned.cuda()
        call = lambda **kw: nrc.context_tree_attention(q, d["cache"], d["tables"], d["ctx_lens"], starts, most,
                                                       tree_mask=mask, max_ctx=max(ctx), **kw)
        poison(T * Hq * 128, T * Hq * 4)
        out, lse = call()
        assert bool((out[~owned] == 0).all()) and bool((lse[~owned] == -math.inf).all())
        if most == max(nodes):
            assert torch.equal(out[owned], want) and torch.equal(lse[owned], want_l)
        given = torch.full_like(out, 5.0)
        same, l2 = call(out=given)
        assert bool((given[~owned] == 5).all()) and torch.equal(given[owned], out[owned]) and torch.equal(l2, lse)
        given = torch.full_like(lse, 6.0)
        o2, same = call(lse=given)
        assert bool((given[~owned] == 6).all()) and torch.equal(given[owned], lse[owned]) and torch.equal(o2, out)


def test_attention_rows_of_ranges_outside(nrc):
    """Ranges of rows outside q write nothing of their own: their rows are rows of no sequence."""
    bt = ref.Batch([20, 30], [3, 6], seed=51)
    d = bt.dev()
    args = lambda starts: (d["q"], d["cache"], d["tables"], d["ctx_lens"],
                           torch.tensor(starts, dtype=torch.int32, device="cuda"), 6)
    want = nrc.context_tree_attention(*args([0, 3, 9]), tree_mask=d["tree_mask"])
    for starts, owned in (([0, 3, 99], slice(0, 3)), ([-2, 3, 9], slice(3, 9)), ([0, 3, 2 ** 31 - 1], slice(0, 3)),
                          ([50, 60, 70], slice(0, 0)), ([-9, -5, -2], slice(0, 0)), ([5, 5, 5], slice(0, 0))):
        poison(9 * 8 * 128, 9 * 8 * 4)
        out, lse = nrc.context_tree_attention(*args(starts), tree_mask=d["tree_mask"])
        rest = torch.ones(9, dtype=torch.bool, device="cuda")
        rest[owned] = False
        assert bool((out[rest] == 0).all()) and bool((lse[rest] == -math.inf).all()), starts
        assert torch.equal(out[owned], want[0][owned]) and torch.equal(lse[owned], want[1][owned]), starts


def test_attention_without_a_sequence(nrc):
    bt = ref.Batch([20, 30], [3, 6], seed=52)
    d = bt.dev()
    poison(9 * 8 * 128, 9 * 8 * 4)
    out, lse = nrc.context_tree_attention(d["q"], d["cache"], d["tables"][:0], d["ctx_lens"][:0], d["q_starts"][:1], 1)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    given = torch.full_like(out, 5.0)
    nrc.context_tree_attention(d["q"], d["cache"], d["tables"][:0], d["ctx_lens"][:0], d["q_starts"][:1], 1, out=given)
    assert bool((given == 5).all())


def test_captured_attention_of_a_padded_batch(nrc):
    """T fixed at capture, sequences' rows moved under it: each replay leaves the rows of nobody at 0 and -inf."""
    bt = ref.Batch([300, 200], [3, 6], seed=53)
    d = bt.dev()
    q = torch.cat([d["q"], d["q"]])
    starts = torch.tensor([0, 3, 9], dtype=torch.int32, device="cuda")
    call = lambda: nrc.context_tree_attention(q, d["cache"], d["tables"], d["ctx_lens"], starts, 6, max_ctx=300)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    for s in ([0, 3, 9], [2, 4, 7], [0, 0, 1], [9, 12, 18]):
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        out.fill_(3.0)
        lse.fill_(3.0)
        g.replay()
        eager = call()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        assert bool((out[:s[0]] == 0).all()) and bool((lse[s[2]:] == -math.inf).all())


def turned(x, pos, table, layout, inverse):
    """The rotation in 64 bits, of a tensor that may carry a graph; rows outside the table as they are."""
    R = table.shape[1]
    row = table[pos.clamp(0, table.shape[0] - 1)][:, None, :]
    c, s = row[..., :R // 2], row[..., R // 2:] * (-1 if inverse else 1)
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if layout == "interleaved" else (x[..., :R // 2], x[..., R // 2:R])
    y, z = a * c - b * s, b * c + a * s
    y = torch.stack([y, z], -1).flatten(-2) if layout == "interleaved" else torch.cat([y, z], -1)
    inside = ((pos >= 0) & (pos < table.shape[0]))[:, None, None]
    return torch.where(inside, torch.cat([y, x[..., R:]], -1), x)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate_carries_the_gradient(nrc, dtype, layout, inverse):
    """Against the formula's gradient in 64 bits and against differences; a padded row's passes through."""
    T, H, d, R = 7, 3, 24, 16
    gen = torch.Generator().manual_seed(54)
    x = torch.randn(T, H, d, generator=gen).to(dtype)
    g = torch.randn(T, H, d, generator=gen).to(dtype)
    pos = torch.randint(0, 40, (T,), generator=gen)
    pos[4] = -1
    table = nrc.rope_table(40, R, dtype=torch.float32, magnitude=1.25)
    table64 = table.double().cpu()
    leaf = x.cuda().requires_grad_()
    y = nrc.rope_rotate(leaf, pos.cuda(), table, layout=layout, inverse=inverse)
    assert y.requires_grad
    y.backward(g.cuda())
    leaf64 = x.double().requires_grad_()
    turned(leaf64, pos, table64, layout, inverse).backward(g.double())
    # two products and sums of FP32 (2^-24 each of the terms' size, up to 2 sqrt(2) x 1.25 g) and half a step of the type
    want = leaf64.grad
    tol = want.abs() * torch.finfo(dtype).eps / 2 + 4 * 2.0 ** -24 * 3.6 * float(g.double().abs().max())
    assert bool(((leaf.grad.double().cpu() - want).abs() <= tol).all())
    assert torch.equal(leaf.grad[4].cpu(), g[4])
    if dtype == torch.float32:
        # the map is linear: differences of its own outputs over steps of 1
        f = lambda t: float((nrc.rope_rotate(t.cuda(), pos.cuda(), table, layout=layout, inverse=inverse).double().cpu()
                             * g.double()).sum())
        for at in ((2, 1, 0), (2, 1, 9), (2, 1, 20), (4, 0, 3)):
            e = torch.zeros_like(x)
            e[at] = 1.0
            assert abs((f(e) - f(-e)) / 2 - float(want[at])) <= 8 * 2.0 ** -24 * float(g.abs().max()) * 1.25
    # a sum's gradient is one value without strides; a second derivative is the rotation again
    leaf.grad = None
    nrc.rope_rotate(leaf, pos.cuda(), table, layout=layout, inverse=inverse).sum().backward()
    ones = nrc.rope_rotate(torch.ones_like(leaf).detach(), pos.cuda(), table, layout=layout, inverse=not inverse)
    assert torch.equal(leaf.grad, ones)
    go = g.cuda().requires_grad_()
    grad, = torch.autograd.grad(nrc.rope_rotate(leaf, pos.cuda(), table, layout=layout, inverse=inverse), leaf, go,
                                create_graph=True)
    again, = torch.autograd.grad(grad, go, x.cuda())
    assert torch.equal(again, nrc.rope_rotate(x.cuda(), pos.cuda(), table, layout=layout, inverse=inverse))


def test_rotate_gradient_is_refused_or_not_wanted(nrc):
    x = torch.randn(5, 2, 64, device="cuda", requires_grad=True)
    pos = torch.arange(5, device="cuda")
    table = nrc.rope_table(10, 64, dtype=torch.float32)
    with pytest.raises(ValueError):
        nrc.rope_rotate(x, pos, table, out=torch.empty_like(x))
    with pytest.raises(ValueError):
        nrc.rope_rotate(x, pos, table, out=x)
    with pytest.raises(ValueError):
        nrc.rope_rotate(x.detach(), pos, table.clone().requires_grad_())
    with torch.no_grad():
        y = nrc.rope_rotate(x, pos, table, out=torch.empty_like(x))
        z = nrc.rope_rotate(x, pos, table.clone().requires_grad_())
    assert not y.requires_grad and torch.equal(y, z)
    assert not nrc.rope_rotate(x.detach(), pos, table).requires_grad
    empty = nrc.rope_rotate(x[:0], pos[:0], table)
    empty.sum().backward()
    assert bool((x.grad == 0).all())


def test_rotate_gradient_captured_and_on_a_stream(nrc):
    gen = torch.Generator().manual_seed(55)
    x = torch.randn(50, 4, 64, generator=gen).cuda().requires_grad_()
    g = torch.randn(50, 4, 64, generator=gen).cuda()
    pos = torch.arange(50, device="cuda")
    table = nrc.rope_table(50, 64)
    step = lambda **kw: torch.autograd.grad(nrc.rope_rotate(x, pos, table, **kw), x, g)[0]
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        on_stream = step()
    s.synchronize()
    assert torch.equal(on_stream, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        g.mul_(2.0)
        out.zero_()
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(out, want * 2.0 ** (k + 1))


@pytest.mark.parametrize("ctx,nodes,H,G", [([100], [1], 2, 4), ([9000], [3], 1, 2), ([700, 30], [40, 9], 1, 4), ([2000], [80], 2, 8)])
def test_attention_in_a_large_padded_buffer(nrc, ctx, nodes, H, G):
    """So many rows of nobody that workgroups of their own fill them: the others' bits are as without."""
    bt = ref.Batch(ctx, nodes, H=H, G=G, seed=56, tree=False)
    d = bt.dev()
    rest = (d["cache"], d["tables"], d["ctx_lens"])
    want, want_l = nrc.context_tree_attention(d["q"], *rest, d["q_starts"], max(nodes), max_ctx=max(ctx))
    for before, behind in ((0, 20000), (20000, 0), (7001, 9000)):
        q = torch.zeros(before + bt.T + behind, H * G, 64, dtype=torch.bfloat16, device="cuda")
        q[before:before + bt.T] = d["q"]
        poison(q.shape[0] * H * G * 128, q.shape[0] * H * G * 4)
        out, lse = nrc.context_tree_attention(q, *rest, d["q_starts"] + before, max(nodes), max_ctx=max(ctx))
        own = slice(before, before + bt.T)
        assert torch.equal(out[own], want) and torch.equal(lse[own], want_l)
        assert bool((out[:before] == 0).all()) and bool((out[before + bt.T:] == 0).all())
        assert bool((lse[:before] == -math.inf).all()) and bool((lse[before + bt.T:] == -math.inf).all())
        given = torch.full_like(out, 5.0)
        _, l2 = nrc.context_tree_attention(q, *rest, d["q_starts"] + before, max(nodes), max_ctx=max(ctx), out=given)
        assert bool((given[:before] == 5).all()) and bool((given[before + bt.T:] == 5).all())
        assert torch.equal(given[own], want) and torch.equal(l2, lse)
