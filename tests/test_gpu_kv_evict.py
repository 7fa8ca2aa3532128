"""context_kv_evict against a plain sort: moved values, so every bit."""

import math

import pytest

import cache_ref as ref
from helpers import to_host

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def make(lens, H=2, bs=16, seed=1, width=None):
    bt = ref.Batch(lens, [0] * len(lens), H=H, block_size=bs, seed=seed, tree=False)
    gen = torch.Generator().manual_seed(seed)
    width = max(max(lens), 1) if width is None else width
    w = torch.exp(2 * torch.randn(len(lens), H, width, generator=gen))
    p = torch.arange(width, dtype=torch.int32).expand(len(lens), H, width).contiguous()
    return dict(cache=bt.cache, tables=bt.tables, lens=bt.ctx_lens, weights=w, positions=p,
                ends=torch.tensor(lens, dtype=torch.int32))


def check(nrc, c, budget, sinks=0, recent=0):
    want = ref.evict(c["cache"], c["tables"], c["lens"], c["weights"], c["positions"], c["ends"], budget, sinks, recent)
    d = {k: v.cuda() for k, v in c.items()}
    got = nrc.context_kv_evict(d["cache"], d["tables"], d["lens"], d["weights"], d["positions"], d["ends"], budget,
                               sinks=sinks, recent=recent)
    torch.cuda.synchronize()
    for name, g, w in zip(("weights", "positions", "lens"), got, want):
        g = g.cpu()
        assert torch.equal(torch.nan_to_num(g.float(), nan=-9.0), torch.nan_to_num(w.float(), nan=-9.0)), name
    assert (to_host(d["cache"]) == to_host(want[3])).all(), "cache"
    return got, d


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 300, 1025, 2049])
@pytest.mark.parametrize("share", [0.02, 0.5, 0.97, 1.0, 1.5])
def test_lengths_and_budgets(nrc, n, share):
    check(nrc, make([n], seed=n), max(1, int(n * share)))


@pytest.mark.parametrize("bs", [1, 3, 16, 24, 64])
def test_block_sizes(nrc, bs):
    check(nrc, make([200, 90, 0, 5], bs=bs, seed=bs), 80, sinks=4, recent=10)


@pytest.mark.parametrize("n,budget", [(5000, 4096), (5000, 10), (17000, 9000), (70000, 30000)])
def test_long_heads(nrc, n, budget):
    """Past what the kernels hold in registers at each size."""
    check(nrc, make([n, n // 3], H=1, seed=n), budget, sinks=4, recent=100)


@pytest.mark.parametrize("n,budget,H", [(8000, 4000, 2), (1500, 750, 260), (12000, 6000, 1), (33000, 32000, 33), (33000, 500, 2), (65536, 32768, 1),
                                        (65537, 1, 2), (140000, 70001, 1)])
def test_lists_of_one_and_of_many_workgroups(nrc, n, budget, H):
    """Each way of selecting: the lists shorter than the array too, of a length that leaves parts empty."""
    c = make([n, n // 2 + 77] if H < 3 else [n], H=H, bs=64, seed=n)
    check(nrc, c, budget, sinks=4, recent=33)
    if H < 3:
        c["lens"][1] = min(budget + 3, n)
        check(nrc, c, budget)


@pytest.mark.parametrize("kind", ["one", "few", "signs", "close", "nan"])
def test_ties_over_many_workgroups(nrc, kind):
    n = 40000
    c = make([n, n - 4097], H=2, bs=64, seed=12)
    gen = torch.Generator().manual_seed(13)
    w = c["weights"]
    if kind == "one":
        w.fill_(0.25)
    elif kind == "few":
        w.copy_(torch.randint(0, 5, w.shape, generator=gen).float())
    elif kind == "signs":
        w.copy_(torch.randint(-2, 3, w.shape, generator=gen).float() * 0.0)
    elif kind == "close":  # differ in the last digit alone, many times each
        w.copy_((torch.randint(0, 700, w.shape, generator=gen).int() + 0x3F800000).view(torch.float32))
    else:
        w[torch.rand(w.shape, generator=gen) < 0.6] = math.nan
    for budget in (1, 9999, 20480, n - 1):
        check(nrc, c, budget, sinks=2, recent=5)


def test_ties_keep_the_first(nrc):
    c = make([500, 500, 500], seed=2)
    c["weights"][0] = 0.0
    c["weights"][1] = torch.randint(0, 3, c["weights"][1].shape, generator=torch.Generator().manual_seed(3)).float()
    c["weights"][2, :, ::2] = -0.0
    c["weights"][2, :, 1::2] = 0.0
    check(nrc, c, 200)
    check(nrc, c, 499, sinks=3, recent=3)


def test_nan_infinities_and_negative_weights(nrc):
    c = make([400], seed=4)
    w = c["weights"]
    w[0, 0, ::3] = math.nan
    w[0, 0, 1::5] = -math.inf
    w[0, 1, ::2] *= -1
    w[0, 1, 7] = math.inf
    w[0, 1, 350] = 1e-42  # subnormal
    check(nrc, c, 150)
    check(nrc, c, 350, recent=20)


def test_more_protected_than_the_budget(nrc):
    check(nrc, make([300, 100], seed=5), 50, sinks=40, recent=60)
    check(nrc, make([300, 100], seed=5), 50, sinks=1000)


def test_positions_decide_protection(nrc):
    """After an eviction the newest tokens sit in holes: their positions keep them."""
    c = make([300], seed=6)
    (w, p, n), d = check(nrc, c, 200, sinks=4, recent=50)
    kept = set(p[0, 0].tolist())
    assert set(range(4)) <= kept and set(range(250, 300)) <= kept
    c2 = dict(cache=d["cache"].cpu(), tables=c["tables"], lens=n.cpu(), weights=w.cpu(), positions=p.cpu(), ends=c["ends"])
    (w2, p2, n2), _ = check(nrc, c2, 120, sinks=4, recent=50)
    kept = set(p2[0, 1].tolist())
    assert set(range(4)) <= kept and set(range(250, 300)) <= kept


def test_heads_choose_for_themselves(nrc):
    (w, p, n), _ = check(nrc, make([256, 256], H=8, seed=7), 64)
    assert not torch.equal(p[0, 0], p[0, 1])


def test_absent_blocks_and_lengths_past_the_arrays(nrc):
    c = make([200, 90], seed=8)
    c["tables"][0, 1] = -1
    c["tables"][0, 9] = c["cache"].shape[0]
    c["lens"][1] = 10 ** 9  # cut to the width, then to the table
    check(nrc, c, 70)
    c["lens"][0] = -5
    check(nrc, c, 70)


def test_strided_values_and_views(nrc):
    c = make([150, 80], H=2, seed=9)
    want = ref.evict(c["cache"], c["tables"], c["lens"], c["weights"], c["positions"], c["ends"], 60, 2, 5)
    nb, H, bs, _ = c["cache"].shape
    pool = torch.zeros(nb, bs, H, 136, dtype=torch.bfloat16, device="cuda")
    view = pool.permute(0, 2, 1, 3)[..., 8:136]
    view.copy_(c["cache"])
    w = torch.zeros(H, 2, 160, device="cuda").permute(1, 0, 2)[:, :, 7:157]
    w.copy_(c["weights"])
    p = torch.zeros(2, H, 151, dtype=torch.int32, device="cuda")[:, :, 1:]
    p.copy_(c["positions"])
    got = nrc.context_kv_evict(view, c["tables"].cuda(), c["lens"].cuda(), w, p, c["ends"].cuda(), 60, sinks=2, recent=5)
    for g, x in zip(got, want):
        assert torch.equal(g.cpu(), x)
    assert (to_host(view) == to_host(want[3])).all()
    assert bool((pool[..., :8] == 0).all())


def test_graph_and_stream(nrc):
    c = make([600, 500], seed=10)
    want = ref.evict(c["cache"], c["tables"], c["lens"], c["weights"], c["positions"], c["ends"], 300, 4, 20)
    d = {k: v.cuda() for k, v in c.items()}
    call = lambda cache, **kw: nrc.context_kv_evict(cache, d["tables"], d["lens"], d["weights"], d["positions"], d["ends"],
                                                    300, sinks=4, recent=20, **kw)
    work = [d["cache"].clone() for _ in range(2)]
    graphs, outs = [], []
    call(d["cache"].clone())
    torch.cuda.synchronize()
    for x in work:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    for _ in range(3):
        for x, g in zip(work, graphs):
            x.copy_(d["cache"])
            g.replay()
            call(d["cache"].clone())
        torch.cuda.synchronize()
        for x, o in zip(work, outs):
            assert (to_host(x) == to_host(want[3])).all()
            assert all(torch.equal(a.cpu(), b) for a, b in zip(o, want))
            o[0].fill_(3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    x = d["cache"].clone()
    s.wait_stream(torch.cuda.current_stream())
    o = call(x, stream=s)
    s.synchronize()
    assert (to_host(x) == to_host(want[3])).all() and all(torch.equal(a.cpu(), b) for a, b in zip(o, want))


def test_refusals(nrc):
    c = make([100, 50], seed=11)
    d = {k: v.cuda() for k, v in c.items()}
    ok = dict(d, budget=40)
    nrc.context_kv_evict(**{**ok, "cache": d["cache"].clone()})
    before = to_host(d["cache"])
    bad = [dict(budget=0), dict(budget=-1), dict(budget=2 ** 33), dict(sinks=-1), dict(recent=-1),
           dict(weights=d["weights"].double()), dict(weights=d["weights"][0]), dict(weights=d["weights"].cpu()),
           dict(positions=d["positions"].long()), dict(positions=d["positions"][:, :, :50]), dict(lens=d["lens"][:1]),
           dict(ends=d["ends"].long()), dict(cache=d["cache"].float()), dict(cache=d["cache"][..., :120]),
           dict(tables=d["tables"].long()), dict(new_weights=torch.empty(2, 2, 39, device="cuda")),
           dict(new_positions=torch.empty(2, 2, 40, device="cuda")), dict(new_lens=torch.empty(2, device="cuda")),
           dict(new_lens=d["lens"]), dict(new_lens=d["ends"]),
           dict(new_weights=d["weights"].view(-1)[:160].view(2, 2, 40))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, nrc.NrcError)):
            nrc.context_kv_evict(**{**ok, **kw})
    assert (to_host(d["cache"]) == before).all()
    # no sequence, no cells
    got = nrc.context_kv_evict(d["cache"], d["tables"][:0], d["lens"][:0], d["weights"][:0], d["positions"][:0],
                               d["ends"][:0], 4)
    assert got[0].shape == (0, 2, 4)
