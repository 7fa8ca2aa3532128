"""The operators around the cache on the ways through their kernels that need large
calls: the received weight's two tiles of keys a wave, split contexts of 17 to 32
rows, capped scores of more than 256 rows, long chains and trees, long tables."""

import math

import pytest

import cache_ref as ref
from test_gpu_rope import frequencies, half_step
from test_gpu_tree_attention import assert_within, check, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def any_mask(bt, seed):
    bt.mask = torch.randint(-2 ** 62, 2 ** 62, bt.mask.shape, generator=torch.Generator().manual_seed(seed))


def spoil(bt, b, node, d, value):
    """Puts value into element d of V of a node, of every head."""
    c = bt.cell(b, bt.ctx[b] + node)
    bt.cache[c[0], :, c[1], 64 + d] = value


def check_odd(nrc, bt, cap=0.0, **kw):
    """check, where V holds infinities and NaN (an element that meets one has no bound)."""
    out, lse, _, _ = run(nrc, bt, softcap=cap, **kw)
    o, l, to, tl = ref.attention(bt, 0.125, cap)
    assert_within(out, o, torch.nan_to_num(to, nan=0.0), "out")
    assert_within(lse, l, tl, "lse")


# ---- received weight ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("ctx,nodes,H,G,blocks,tree", [
    ([0, 1, 31, 64, 65, 127, 150, 3] * 2, [20, 1, 7, 16, 13, 0, 20, 9] * 2, 8, 5, 5, True),  # 100 rows, short and ragged
    ([2000, 700, 513], [40, 33, 0], 2, 3, 90, True),                                         # whole tiles of context
    ([900, 256], [70, 1], 1, 1, 260, False),                                                 # a chain, one head
    ([300] * 9, [1] * 9, 8, 8, 8, False),                                                    # one token each
])
def test_mass_of_two_tiles_a_wave(nrc, cap, ctx, nodes, H, G, blocks, tree):
    """Enough keys that a wave takes 64 of them: 256 to a workgroup, two workgroups a CU and more."""
    bt = ref.Batch(ctx, nodes, H=H, G=G, seed=60 + G, tree=tree)
    width = blocks * 256 - 77
    assert -(-width // 256) * H * len(ctx) >= 2 * cus()
    if tree:
        any_mask(bt, 61)
    bt.tables[-2, 0], bt.tables[0, -1] = -1, bt.nb
    o, l, _, _ = ref.attention(bt, cap=cap)
    d = bt.dev()
    args = (d["q"], d["cache"], d["tables"], d["ctx_lens"], d["q_starts"], l.float().cuda(), d["max_nodes"])
    w = torch.rand(bt.B, H, width, generator=torch.Generator().manual_seed(62))
    for weights, decay in ((None, 1.0), (w, 0.75)):
        want, tol = ref.mass(bt, l.float(), width, weights, decay, cap=cap)
        given = None if weights is None else weights.cuda()
        got = nrc.context_attention_mass(*args, tree_mask=d["tree_mask"], softcap=cap, weights=given, decay=decay, width=width)
        assert_within(got, want, tol, "mass")
        if given is not None:
            nrc.context_attention_mass(*args, tree_mask=d["tree_mask"], softcap=cap, weights=given, decay=decay, out=given)
            assert torch.equal(given, got)


def test_mass_of_one_and_of_two_tiles_agree(nrc):
    """The same cells in a narrow call and in one wide enough for two tiles a wave: the same bits."""
    bt = ref.Batch([600, 95], [25, 40], H=2, G=4, seed=63)
    out, lse, args, d = run(nrc, bt)
    wide = 128 * 256
    assert wide // 256 * 4 >= 2 * cus() > 3 * 4
    few = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], width=650)
    many = nrc.context_attention_mass(*args, lse, d["max_nodes"], tree_mask=d["tree_mask"], width=wide)
    assert torch.equal(many[:, :, :650], few) and bool((many[:, :, 650:] == 0).all())


def test_mass_of_two_tiles_with_scores_past_the_exponent(nrc):
    bt = ref.Batch([90, 33] * 8, [9, 6] * 8, H=8, G=4, seed=64, tree=False)
    q, k = bt.q[..., :1].clone(), bt.cache[..., :1].clone()
    bt.q.zero_()
    bt.cache[..., :64] = 0
    bt.q[..., :1], bt.cache[..., :1] = q * 1e10, k * 1e10
    out, lse, args, d = run(nrc, bt)
    m = nrc.context_attention_mass(*args, lse, d["max_nodes"], width=1024)
    assert 4 * 8 * 16 >= 2 * cus()
    few = torch.cat([nrc.context_attention_mass(q2, d["cache"], d["tables"][2 * i:2 * i + 2], d["ctx_lens"][2 * i:2 * i + 2],
                                                torch.tensor([0, 9, 15], dtype=torch.int32, device="cuda"),
                                                lse[15 * i:15 * i + 15], 9, width=1024)
                     for i, q2 in enumerate(d["q"].split(15))])
    # (no bound on the weights themselves: lse is FP32, so at scores of 2^63 it lies up to 2^39 from its exact value, and
    # e^(score - lse) anywhere from 0 to infinity)
    assert bool((m >= 0).all()) and torch.equal(m, few)


# ---- attention, 17 to 32 rows a head ------------------------------------------------------------------------------


@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("H,G,nodes,bs,tree", [(1, 4, [7, 5], 16, True), (2, 2, [13, 1], 24, True), (1, 1, [32, 17], 48, False),
                                               (1, 5, [6, 0], 3, True)])
def test_split_contexts_of_17_to_32_rows(nrc, cap, H, G, nodes, bs, tree):
    ctx = [5000, 1300]
    assert 16 < max(nodes) * G <= 32
    bt = ref.Batch(ctx, nodes, H=H, G=G, block_size=bs, seed=65 + bs, tree=tree)
    assert nrc._load().nrc_context_tree_attention_workspace_bytes(2, bt.T, H * G, H, bt.max_nodes, 5000) > 0
    check(nrc, bt, cap=cap, max_ctx=5000, mass=False)
    # blocks that are not there, in the middle of a split and at its end
    for blk in (1, 700 // bs, 701 // bs + 1, 4000 // bs, bt.tables.shape[1] - 1):
        bt.tables[0, blk] = -1
    check(nrc, bt, cap=cap, max_ctx=5000, mass=False)


@pytest.mark.parametrize("nodes,G", [(6, 2), (14, 2), (8, 4)])
@pytest.mark.parametrize("ctx", [37, 3000])
def test_odd_values_of_nodes_few_rows(nrc, nodes, G, ctx):
    """Infinities and NaN in V of nodes that some rows see."""
    for value in (math.nan, math.inf, -math.inf):
        bt = ref.Batch([ctx, 20], [nodes, 3], H=2, G=G, seed=66)
        spoil(bt, 0, 3, 11, value)
        spoil(bt, 1, 1, 60, value)
        check_odd(nrc, bt, max_ctx=ctx)
        check_odd(nrc, bt, cap=20.0, max_ctx=ctx)
    bt = ref.Batch([ctx, 20], [nodes, 3], H=2, G=G, seed=66)
    spoil(bt, 0, 2, 5, math.inf)  # both in one element: NaN for the rows that see the two
    spoil(bt, 0, 4, 5, -math.inf)
    any_mask(bt, 67)
    check_odd(nrc, bt, max_ctx=ctx)


@pytest.mark.parametrize("nodes", [3, 14, 40])
@pytest.mark.parametrize("at", [5, 98, 120])
def test_infinities_in_the_context(nrc, nodes, at):
    """V of a context key, in a whole tile and in the one it shares with nodes: every row sees it."""
    bt = ref.Batch([123], [nodes], H=1, G=2, seed=68, q_scale=1.0)
    c = bt.cell(0, at)
    bt.cache[c[0], 0, c[1], 64 + 9] = math.inf
    bt.cache[c[0], 0, c[1], 64 + 33] = math.nan
    check_odd(nrc, bt)


# ---- attention, more than 256 rows of capped scores ---------------------------------------------------------------


@pytest.mark.parametrize("ctx", [[1000, 600], [100, 0], [6000, 3]])
@pytest.mark.parametrize("G,nodes", [(4, [70, 66]), (5, [100, 3]), (1, [300, 257])])
def test_capped_trees_of_many_rows(nrc, ctx, G, nodes):
    assert max(nodes) * G > 256
    bt = ref.Batch(ctx, nodes, H=1, G=G, seed=69)
    check(nrc, bt, cap=25.0, max_ctx=max(ctx), mass=False)
    any_mask(bt, 70)
    for blk in (0, 20, 21, bt.tables.shape[1] - 2):
        if blk < bt.tables.shape[1]:
            bt.tables[0, blk] = -1
    check(nrc, bt, cap=25.0, max_ctx=max(ctx), mass=False)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cap", [0.0, 25.0])
def test_odd_values_of_nodes_many_rows(nrc, value, cap):
    bt = ref.Batch([1000, 600], [70, 66], H=1, G=4, seed=71)
    for b, node, d in ((0, 5, 9), (0, 65, 33), (1, 40, 63), (1, 41, 0)):
        spoil(bt, b, node, d, value)
    any_mask(bt, 72)
    check_odd(nrc, bt, cap=cap)


# ---- long chains and trees ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("cap", [0.0, 25.0])
@pytest.mark.parametrize("ctx,nodes,H,G,tree", [([500, 90], [700, 300], 1, 2, True), ([0, 1000], [1500, 2], 1, 1, False),
                                                ([129, 0, 64], [513, 128, 1], 2, 3, False), ([3000], [1025], 1, 1, True)])
def test_long_chains_and_trees(nrc, cap, ctx, nodes, H, G, tree):
    """Several blocks of rows, whole tiles of nodes, masks of many words; one sequence's rows split over workgroups."""
    bt = ref.Batch(ctx, nodes, H=H, G=G, seed=73, tree=tree)
    check(nrc, bt, cap=cap, max_ctx=max(ctx))


def test_a_chain_of_thousands(nrc):
    bt = ref.Batch([77], [4100], H=1, G=1, seed=74, tree=False)
    check(nrc, bt)


def test_masks_of_the_most_words(nrc):
    """1024 words a row, the words past the nodes set too."""
    bt = ref.Batch([50, 10], [9, 130], H=1, G=2, seed=75, words=1024)
    any_mask(bt, 76)
    check(nrc, bt)


# ---- tables -------------------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,width,count,start,scaling,run", [
    (64, 64, 65536 + 4471, 12345, "base", 16), (64, 70, 70007, 2 ** 28 - 70007, "ramp", 16), (6, 64, 66003, 1, "none", 16),
    (128, 130, 9001, 99990, "linear", 4), (256, 256, 2111, 0, "bands", 2), (64, 64, 33003, 7, "ramp", 8)])
def test_table_of_runs(nrc, dtype, R, width, count, start, scaling, run):
    """Several positions to a sincos, turned on step by step, the last run short."""
    half = width // 2
    r = 16
    while r > 1 and count * half // r < cus() * 512:
        r //= 2
    assert r == run and count % run
    got = nrc.rope_table(count, R, base=500000.0, scaling=scaling, factor=8.0, original_max=8192, low=1.0, high=32.0,
                         magnitude=1.1, width=width, start=start, dtype=dtype)
    a = torch.arange(start, start + count, dtype=torch.float64)[:, None] * frequencies(R, 500000.0, scaling, 8.0, 8192, 1.0, 32.0)
    want = torch.zeros(count, width, dtype=torch.float64)
    want[:, R // 2:half] = 1.0
    want[:, :R // 2], want[:, half:half + R // 2] = 1.1 * torch.cos(a), 1.1 * torch.sin(a)
    # an angle of up to start + count radians is off by 4 roundings of 2^-53 in its frequency (pow, the scaling) and one in
    # the product, on both sides; the cos and sin of a step by 2^-53 and each of the run's 16 steps by 3 roundings of
    # values up to 1; one rounding to the type, after one to FP32
    angle = (start + count) * 10 * 2.0 ** -53 + 16 * 4 * 2.0 ** -53
    tol = want.abs() * (half_step(dtype) + 2.0 ** -24) + 1.1 * angle
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


def whole_reference(q, run, ctx, words, step=2048):
    """One sequence of one head in 64 bits on the GPU, some rows at a time, with cache_ref's bounds (attention's, and of
    every key's received weight): out, lse, mass of the keys, and their bounds. run [keys, 128]; words: the mask or None."""
    n, keys = q.shape[0], run.shape[0]
    k, v = run[:, :64].double(), run[:, 64:].double()
    kt, ka, va = k.T.contiguous(), k.abs().T.contiguous(), v.abs()
    at = torch.arange(keys, device="cuda") - ctx
    got = [torch.zeros(n, 64, dtype=torch.float64), torch.zeros(n, dtype=torch.float64), torch.zeros(n, 64, dtype=torch.float64),
           torch.zeros(n, dtype=torch.float64)]
    mass, bound = torch.zeros(keys, dtype=torch.float64, device="cuda"), torch.zeros(keys, dtype=torch.float64, device="cuda")
    for lo in range(0, n, step):
        qs = q[lo:lo + step].double()
        s = torch.mm(qs, kt) * 0.125
        e = 64 * 2.0 ** -23 * torch.mm(qs.abs(), ka) * 0.125 + s.abs() * 2.0 ** -21
        if words is None:
            sees = at[None, :] <= torch.arange(lo, lo + qs.shape[0], device="cuda")[:, None]
        else:
            w = words[lo:lo + step].gather(1, (at.clamp(min=0) // 64).expand(qs.shape[0], -1))
            sees = ((w >> (at.clamp(min=0) % 64)) & 1 == 1) | (at < 0)
        s = s.masked_fill(~sees, -math.inf)
        l = torch.logsumexp(s, 1)
        p = torch.exp(s - l[:, None])
        o, A = torch.mm(p, v), torch.mm(p, va)
        eps = e.masked_fill(~sees, 0.0).amax(1) + 2.0 ** -22 + keys * 2.0 ** -24
        part = (o, l, o.abs() * 2.0 ** -8 + (2 * eps[:, None] + 2.0 ** -8) * A * 1.01, eps * 1.01 + (l.abs() + 24) * 3 * 2.0 ** -24)
        for g, x in zip(got, part):
            g[lo:lo + step] = x.cpu()
        # with lse rounded to FP32, as the call takes it
        d = torch.where(sees, s - l.float().double()[:, None], 0.0)
        w = torch.where(sees, torch.exp(d), 0.0)
        mass += w.sum(0)
        bound += (w * (e + d.abs() * 3 * 2.0 ** -24 + 2.0 ** -22 + n * 2.0 ** -24) * 1.01).sum(0)
    return (*got, mass.cpu(), (bound + mass.abs() * 2.0 ** -22 + 1e-37).cpu())


@pytest.mark.parametrize("nodes,ctx,tree", [(65535, 1001, False), (20011, 300, True)])
def test_the_longest_chains_and_trees(nrc, nodes, ctx, tree):
    gen = torch.Generator(device="cuda").manual_seed(77)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    keys, bs = ctx + nodes, 16
    blocks = -(-keys // bs)
    q = (2 * normal(nodes, 1, 64)).to(torch.bfloat16)
    cache = normal(blocks + 2, 1, bs, 128).to(torch.bfloat16)
    tables = torch.randperm(blocks + 2, generator=gen, device="cuda")[None, :blocks].int()
    words = None
    if tree:  # (a node here sees half of all)
        words = torch.randint(-2 ** 62, 2 ** 62, (nodes, (nodes + 63) // 64 + 1), generator=gen, device="cuda")
    run_of = cache[tables[0].long()].transpose(1, 2).reshape(-1, 128)[:keys]
    o, l, to, tl, m, tm = whole_reference(q[:, 0], run_of, ctx, words)
    args = (q, cache, tables, torch.tensor([ctx], dtype=torch.int32, device="cuda"),
            torch.tensor([0, nodes], dtype=torch.int32, device="cuda"))
    out, lse = nrc.context_tree_attention(*args, nodes, tree_mask=words)
    assert_within(out[:, 0], o, to, "out")
    assert_within(lse[:, 0], l, tl, "lse")
    got = nrc.context_attention_mass(*args, l.float().cuda()[:, None].contiguous(), nodes, tree_mask=words, width=keys)
    assert_within(got[0, 0], m, tm, "mass")
