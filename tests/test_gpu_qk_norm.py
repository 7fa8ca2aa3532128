"""qk_norm_rotate and its gradient against 64-bit references."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from draft_ref import norm_rotate, norm_rotate_grad, turn  # noqa: E402

TYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1, 1, 64, 64), (5, 3, 2, 64, 64), (17, 24, 3, 128, 64), (3, 5, 1, 80, 48), (33, 1, 7, 96, 96), (2, 7, 2, 66, 34),
          (130, 64, 8, 64, 16), (7, 2, 2, 256, 256), (9, 3, 3, 2, 2), (4, 2, 5, 37, 20)]


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def dev(t):
    return None if t is None else t.cuda()


def within(got, want, tol):
    got = got.double().cpu()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])


def inputs(T, Hq, Hk, d, R, dtype, wtype, seed, table=torch.float32):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)
    w = [None, None] if wtype is None else [(1 + 0.3 * n(d)).to(wtype) for _ in range(2)]
    pos = torch.randint(0, 300, (T,), generator=gen)
    angle = torch.arange(300)[:, None] * 10000.0 ** (-torch.arange(R // 2) / (R / 2))
    return dict(q=(2 * n(T, Hq, d)).to(dtype), k=n(T, Hk, d).to(dtype), pos=pos,
                cs=torch.cat([angle.cos(), angle.sin()], 1).to(table), w=w, gq=n(T, Hq, d).to(dtype), gk=n(T, Hk, d).to(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("wtype", [None, torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hk,d,R", SHAPES)
def test_forward_and_gradient(nrc, dtype, layout, wtype, T, Hq, Hk, d, R):
    table = torch.bfloat16 if T % 2 else torch.float32
    i = inputs(T, Hq, Hk, d, R, dtype, wtype, T * 100 + d, table)
    args = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    out = nrc.qk_norm_rotate(*args, eps=1e-5, layout=layout)
    back = nrc.qk_norm_rotate_grad(dev(i["gq"]), dev(i["gk"]), *args, eps=1e-5, layout=layout)
    for part, (x, g, w) in enumerate(((i["q"], i["gq"], i["w"][0]), (i["k"], i["gk"], i["w"][1]))):
        within(out[part], *norm_rotate(x, w, i["pos"], i["cs"], layout, 1e-5))
        dx, tol, dw, dw_tol = norm_rotate_grad(g, x, w, i["pos"], i["cs"], layout, 1e-5)
        within(back[part], dx, tol)
        if w is None:
            assert back[2 + part] is None
        else:
            assert back[2 + part].dtype == w.dtype
            within(back[2 + part], dw, dw_tol)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_gradient_against_differences(nrc, layout):
    """The kernel's gradients against central differences of the 64-bit formula along random directions: h^2 times
    its third derivative (below 100 here) and 2^-52 / h of the values are off."""
    i = inputs(6, 3, 2, 64, 32, torch.float32, torch.float32, 5)
    args = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    back = [t.double().cpu() for t in nrc.qk_norm_rotate_grad(dev(i["gq"]), dev(i["gk"]), *args, layout=layout)]
    gen = torch.Generator().manual_seed(9)
    h = 1e-5
    for part, (x, g, w) in enumerate(((i["q"], i["gq"], i["w"][0]), (i["k"], i["gk"], i["w"][1]))):
        def f(x, w):
            n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
            return float((turn(n, i["pos"], i["cs"], layout)[0] * g.double()).sum())
        x, w = x.double(), w.double()
        _, tx, _, tw = norm_rotate_grad(g, i["qk"[part]], i["w"][part], i["pos"], i["cs"], layout, 1e-6)
        for _ in range(4):
            ux, uw = torch.randn(x.shape, generator=gen).double(), torch.randn(w.shape, generator=gen).double()
            slope = (f(x + h * ux, w) - f(x - h * ux, w)) / (2 * h)
            assert abs(slope - float((back[part] * ux).sum())) <= float((tx * ux.abs()).sum()) + 1e-5
            slope = (f(x, w + h * uw) - f(x, w - h * uw)) / (2 * h)
            assert abs(slope - float((back[2 + part] * uw).sum())) <= float((tw * uw.abs()).sum()) + 1e-5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_views_in_place_and_unaligned(nrc, dtype, layout):
    """Queries, keys (and values) side by side in one tensor's rows, in place; views off by an element."""
    gen = torch.Generator().manual_seed(3)
    T, Hq, Hk, d = 11, 4, 2, 64
    wide = torch.randn(T, (Hq + 2 * Hk) * d + 1, generator=gen).to(dtype).cuda()
    pos = torch.randint(0, 50, (T,), generator=gen).cuda()
    cs = nrc.rope_table(50, d, dtype=torch.float32)
    for first in (0, 1):
        row = wide[:, first:first + (Hq + 2 * Hk) * d].clone() if first == 0 else wide[:, 1:]
        q, k, v = (row[:, a * d:b * d].unflatten(1, (-1, d)) for a, b in ((0, Hq), (Hq, Hq + Hk), (Hq + Hk, Hq + 2 * Hk)))
        kept, k0 = v.clone(), k.clone()
        want = nrc.qk_norm_rotate(q.contiguous(), k.contiguous(), pos, cs, layout=layout)
        got = nrc.qk_norm_rotate(q, k, pos, cs, layout=layout, out_q=q, out_k=k)
        assert got[0] is q and got[1] is k
        # the same arithmetic, summed in another order where the accesses are single elements: a step of the type
        for a, b in zip(got, want):
            assert bool(((a.float() - b.float()).abs() <= b.float().abs() * 2 * torch.finfo(dtype).eps + 1e-5).all())
        assert torch.equal(v, kept)
        assert not torch.equal(k, k0)


def test_heads_before_rows(nrc):
    """[H, T, d] in memory."""
    i = inputs(9, 4, 2, 64, 64, torch.bfloat16, torch.bfloat16, 8)
    flip = lambda t: dev(t).transpose(0, 1).contiguous().transpose(0, 1)
    plain = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    turned = [flip(i["q"]), flip(i["k"])] + plain[2:]
    for a, b in zip(nrc.qk_norm_rotate(*plain), nrc.qk_norm_rotate(*turned)):
        assert torch.equal(a, b)
    for a, b in zip(nrc.qk_norm_rotate_grad(dev(i["gq"]), dev(i["gk"]), *plain),
                    nrc.qk_norm_rotate_grad(flip(i["gq"]), flip(i["gk"]), *turned)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,R", [(64, 64), (66, 34)])
def test_rows_outside_the_table(nrc, d, R):
    i = inputs(6, 3, 2, d, R, torch.bfloat16, torch.bfloat16, 4)
    q, k, pos, cs, qw, kw = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    pos[1], pos[4] = -1, 300
    outside = torch.tensor([1, 4]).cuda()
    q[1, 0, 0] = math.nan
    oq, ok = nrc.qk_norm_rotate(q, k, pos, cs, qw, kw)
    assert torch.equal(oq[outside].view(torch.int16), q[outside].view(torch.int16)) and torch.equal(ok[outside], k[outside])
    gq, gk = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    nrc.qk_norm_rotate(q, k, pos, cs, qw, kw, out_q=gq, out_k=gk)
    assert bool((gq[outside] == 7).all()) and bool((gk[outside] == 7).all())
    rest = torch.tensor([0, 2, 3, 5]).cuda()
    assert torch.equal(gq[rest], oq[rest]) and torch.equal(gk[rest], ok[rest])
    # the gradient passes, and the gains get nothing from these rows (a NaN among them)
    dq, dk, dqw, dkw = nrc.qk_norm_rotate_grad(dev(i["gq"]), dev(i["gk"]), q, k, pos, cs, qw, kw)
    assert torch.equal(dq[outside], dev(i["gq"])[outside]) and torch.equal(dk[outside], dev(i["gk"])[outside])
    r = rest.cpu()
    for got, x, g, w in ((dqw, i["q"], i["gq"], i["w"][0]), (dkw, i["k"], i["gk"], i["w"][1])):
        _, _, dw, tol = norm_rotate_grad(g[r], x[r], w, i["pos"][r], i["cs"], "interleaved", 1e-6)
        within(got, dw, tol)


def test_special_values(nrc):
    """A zero head gives zeros (eps 0: NaN), a NaN or infinity stays within its head, large values do not overflow
    before the norm does."""
    cs = nrc.rope_table(8, 64, dtype=torch.float32)
    x = torch.randn(4, 3, 64, generator=torch.Generator().manual_seed(1))
    x[0, 0], x[1, 1, 5], x[2, 2, 7] = 0.0, math.nan, math.inf
    x[3, 0] *= 1e15
    pos = torch.tensor([1, 2, 3, 4])
    out, none = nrc.qk_norm_rotate(x.cuda(), None, pos.cuda(), cs)
    assert none is None
    assert bool((out[0, 0] == 0).all()) and bool(out[1, 1].isnan().all()) and bool(out[2, 2].isnan().any())
    ok = torch.ones(4, 3, dtype=torch.bool)
    ok[1, 1] = ok[2, 2] = False
    want, tol = norm_rotate(x, None, pos, cs.cpu(), "interleaved", 1e-6)
    got = out.double().cpu()
    assert bool(((got - want).abs() <= tol)[ok].all())
    zero, _ = nrc.qk_norm_rotate(x.cuda(), None, pos.cuda(), cs, eps=0.0)
    assert bool(zero[0, 0].isnan().all())


def test_no_rows_and_no_keys(nrc):
    cs = nrc.rope_table(8, 64)
    e = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones(64, dtype=torch.float32, device="cuda")
    q, k = nrc.qk_norm_rotate(e, e, pos, cs, w, w)
    assert q.shape == e.shape and k.shape == e.shape
    dq, dk, dw, none = nrc.qk_norm_rotate_grad(e, None, e, None, pos, cs, w)
    assert dq.shape == e.shape and dk is None and none is None and bool((dw == 0).all())


def test_many_rows_are_deterministic(nrc):
    """Enough heads for several of each workgroup's lanes, odd numbers of them; two runs give the same bits."""
    i = inputs(4099, 23, 3, 64, 64, torch.bfloat16, torch.float32, 2)
    args = [dev(t) for t in (i["gq"], i["gk"], i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    first = nrc.qk_norm_rotate_grad(*args, layout="half")
    second = nrc.qk_norm_rotate_grad(*args, layout="half")
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    for part, (x, g, w) in enumerate(((i["q"], i["gq"], i["w"][0]), (i["k"], i["gk"], i["w"][1]))):
        dx, tol, dw, dw_tol = norm_rotate_grad(g, x, w, i["pos"], i["cs"], "half", 1e-6)
        within(first[part], dx, tol)
        within(first[2 + part], dw, dw_tol)


def test_autograd(nrc):
    """Inputs and gains that require grad, a broadcast gradient (of a sum), only some of them, under no_grad."""
    i = inputs(12, 4, 2, 64, 32, torch.float32, torch.float32, 6)
    q, k, pos, cs, qw, kw = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    leaves = [t.requires_grad_() for t in (q, k, qw, kw)]
    oq, ok = nrc.qk_norm_rotate(q, k, pos, cs, qw, kw, layout="half")
    grads = torch.autograd.grad((oq.sum() + (ok * ok).sum()), leaves)
    with torch.no_grad():
        pq, pk = nrc.qk_norm_rotate(q, k, pos, cs, qw, kw, layout="half")
        assert not pq.requires_grad and torch.equal(pq, oq) and torch.equal(pk, ok)
        want = nrc.qk_norm_rotate_grad(torch.ones_like(pq), 2 * pk, q, k, pos, cs, qw, kw, layout="half")
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    # one output alone; gains alone
    oq, _ = nrc.qk_norm_rotate(q.detach(), k.detach(), pos, cs, qw, kw)
    (gw,) = torch.autograd.grad(oq.square().sum(), qw)
    assert bool(gw.isfinite().all())
    half = nrc.qk_norm_rotate(q.detach().half().requires_grad_(), None, pos, cs)[0]
    assert half.dtype == torch.float16 and half.requires_grad
    with pytest.raises(ValueError, match="no outputs"):
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=torch.empty_like(q), out_k=torch.empty_like(k))
    with pytest.raises(ValueError, match="detach"):
        nrc.qk_norm_rotate(q, k, pos, cs.clone().requires_grad_())


def test_graph_and_streams(nrc):
    i = inputs(40, 8, 2, 64, 64, torch.bfloat16, torch.float32, 7)
    args = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    gq, gk = dev(i["gq"]), dev(i["gk"])
    want = nrc.qk_norm_rotate(*args) + nrc.qk_norm_rotate_grad(gq, gk, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nrc.qk_norm_rotate(*args, stream=side) + nrc.qk_norm_rotate_grad(gq, gk, *args, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = nrc.qk_norm_rotate(*args) + nrc.qk_norm_rotate_grad(gq, gk, *args)
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, want):
            assert torch.equal(a, b)
        nrc.qk_norm_rotate_grad(gq, gk, *args)


def test_refusals(nrc):
    i = inputs(4, 2, 2, 64, 64, torch.bfloat16, torch.bfloat16, 7)
    q, k, pos, cs, qw, kw = [dev(t) for t in (i["q"], i["k"], i["pos"], i["cs"], *i["w"])]
    for bad in (dict(q=q.cpu()), dict(q=q.double()), dict(k=k.float()), dict(k=k[:3]), dict(k=k[..., :32]),
                dict(pos=pos.int()), dict(pos=pos[:3]), dict(pos=pos.cpu()), dict(cs=cs.half()), dict(cs=cs[:, ::2]),
                dict(qw=qw[:32]), dict(qw=qw.double()), dict(kw=kw.cpu()), dict(layout="other"), dict(q=q[0])):
        a = dict(q=q, k=k, pos=pos, cs=cs, qw=qw, kw=kw, layout="half", **{})
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            nrc.qk_norm_rotate(a["q"], a["k"], a["pos"], a["cs"], a["qw"], a["kw"], layout=a["layout"])
    with pytest.raises(ValueError):
        nrc.qk_norm_rotate(q, None, pos, cs, qw, kw)
    with pytest.raises(ValueError):
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=torch.empty_like(q))
    with pytest.raises(nrc.NrcError, match="apart"):
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=k, out_k=torch.empty_like(k))
    with pytest.raises(nrc.NrcError, match="overlap"):
        nrc.qk_norm_rotate(q, k, pos, cs, out_q=torch.empty_like(q[:1]).expand(4, -1, -1), out_k=torch.empty_like(k))
    with pytest.raises(nrc.NrcError):
        nrc.qk_norm_rotate(q, k, pos, cs, eps=-1.0)
    with pytest.raises(ValueError):
        nrc.qk_norm_rotate_grad(q[:, :1], k, q, k, pos, cs)
