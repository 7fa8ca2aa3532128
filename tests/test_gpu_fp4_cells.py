"""context_fp4_store and context_fp4_load against the definition of the cells."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from draft_ref import STEPS, fp4_groups, fp4_values  # noqa: E402


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def caches(nrc, L, blocks, H, bs, fill=0xA5):
    shape = (blocks, H, nrc.fp4_page_bytes(bs))
    return torch.full(shape if L is None else (L, *shape), fill, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("L,T,H,bs", [(None, 1, 1, 1), (1, 5, 2, 16), (4, 33, 8, 16), (3, 70, 3, 24), (2, 129, 1, 5), (6, 64, 16, 64)])
@pytest.mark.parametrize("per_layer", [False, True])
def test_round_trip(nrc, L, T, H, bs, per_layer):
    if L is None and per_layer:
        pytest.skip("one layer")
    gen = torch.Generator().manual_seed(T * 31 + bs)
    blocks = T // bs + 3
    n = 1 if L is None else L
    kv = (torch.randn(n, T, 2, H, 64, generator=gen) * torch.exp(2 * torch.randn(n, T, 2, H, 1, generator=gen))).bfloat16()
    lists = [torch.randperm(blocks * bs, generator=gen)[:T] for _ in range(n if per_layer else 1)]
    for s in lists:
        s[::7] = -1
        if T > 3:
            s[3] = blocks * bs  # past the cache
    slots = torch.stack(lists) if per_layer else lists[0]
    c = caches(nrc, L, blocks, H, bs)
    d = kv.cuda()
    k, v = (d[:, :, i] if L is not None else d[0, :, i] for i in range(2))
    nrc.context_fp4_store(k, v, slots.cuda(), c)
    got = nrc.context_fp4_load(c, slots.cuda())
    live = ((slots >= 0) & (slots < blocks * bs)).expand(n, T)
    for part in range(2):
        want = torch.where(live[:, :, None, None], fp4_values(kv[:, :, part]), 0.0)
        g = got[part].double().cpu()
        assert torch.equal(g if L is not None else g[None], want)
    # bytes of the cells that no slot names stay as they were
    pages = c.cpu() if L is not None else c.cpu()[None]
    for l in range(n):
        s = lists[l if per_layer else 0]
        s = s[(s >= 0) & (s < blocks * bs)]
        used = torch.zeros(blocks, bs, dtype=torch.bool)
        used[s // bs, s % bs] = True
        for first, width in ((0, 32), (32 * bs, 32), (64 * bs, 4)):
            run = pages[l, :, :, first:first + width * bs].unflatten(-1, (bs, width)).transpose(1, 2)
            assert bool((run[~used] == 0xA5).all())
        assert bool((pages[l, :, :, 68 * bs:] == 0xA5).all())
    # given outputs: rows without a cell stay
    mine = [torch.full(t.shape, 3.0, dtype=torch.bfloat16, device="cuda") for t in got]
    nrc.context_fp4_load(c, slots.cuda(), *mine)
    mask = live.cuda() if L is not None else live[0].cuda()
    for m, g in zip(mine, got):
        assert torch.equal(m[mask], g[mask]) and bool((m[~mask] == 3).all())


def test_every_value_at_every_scale(nrc):
    """All finite bf16 values, each as its group's largest and beside larger ones: codes and scale bytes."""
    bits = torch.arange(65536, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16)
    x = x[x.isfinite()]
    n = x.numel()
    rows = torch.zeros(n, 1, 64, dtype=torch.bfloat16)
    rows[:, 0, 0] = x
    rows[:, 0, 17] = x / 2  # (exact but for the least subnormals)
    rows[:, 0, 30] = -x
    # next to a larger one, 1 to 32 times and more as large
    gen = torch.Generator().manual_seed(1)
    scale = torch.exp2(torch.randint(0, 6, (n,), generator=gen).float()) * (1 + torch.rand(n, generator=gen))
    big = (x.float() * scale).clamp(-3e38, 3e38).bfloat16()
    rows[:, 0, 32], rows[:, 0, 63] = x, big
    c = caches(nrc, None, n, 1, 1)
    slots = torch.arange(n).cuda()
    nrc.context_fp4_store(rows.cuda(), rows.flip(-1).cuda(), slots, c)
    k, v = nrc.context_fp4_load(c, slots)
    want = fp4_values(rows)
    assert torch.equal(k.double().cpu(), want)
    assert torch.equal(v.double().cpu(), fp4_values(rows.flip(-1)))
    code, e = fp4_groups(rows.double().unflatten(-1, (2, 32)))
    page = c.cpu()[:, 0]
    assert torch.equal(page[:, 64:66].long(), e[:, 0] + 127)
    assert torch.equal((page[:, 0] & 7).long(), code[:, 0, 0, 0])
    # the largest of a group lies in (3, 6] times its power of two (the least with which it is at most 6), between the
    # values 3, 4 and 6: off by 1/2 at most below 4 (at 3.5, a seventh of it), by 1 at most above (at 5, a fifth)
    sound = x.abs().double() >= 2.0 ** -118
    sound &= x.abs().double() <= 6 * 2.0 ** 125
    assert bool(((k[:, 0, 0].double().cpu() - x.double()).abs() <= x.double().abs() / 5)[sound].all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", [0, 31, 32, 63])
@pytest.mark.parametrize("part", [0, 1])
def test_infinities_and_nan_make_the_cell_nan(nrc, bad, where, part):
    kv = torch.randn(3, 2, 2, 64, generator=torch.Generator().manual_seed(2)).bfloat16()  # rows, K and V, heads
    kv[1, part, 1, where] = bad
    c = caches(nrc, None, 2, 2, 4)
    slots = torch.tensor([5, 2, 0]).cuda()
    d = kv.cuda()
    nrc.context_fp4_store(d[:, 0], d[:, 1], slots, c)
    k, v = nrc.context_fp4_load(c, slots)
    assert bool((k[1, 1].view(torch.int16) == 0x7FC0).all()) and bool((v[1, 1].view(torch.int16) == 0x7FC0).all())
    k[1, 1] = v[1, 1] = kv[1, :, 1] = 0
    assert torch.equal(k.double().cpu(), fp4_values(kv[:, 0])) and torch.equal(v.double().cpu(), fp4_values(kv[:, 1]))
    page = c.cpu()[0, 1]
    assert bool((page[64 * 4 + 8:64 * 4 + 12] == 255).all())


def test_strided_caches_and_rows(nrc):
    """Pages inside wider ones, heads before blocks, rows of a wider tensor, heads before rows."""
    gen = torch.Generator().manual_seed(4)
    T, H, bs, blocks = 21, 3, 8, 4
    page = nrc.fp4_page_bytes(bs)
    kv = torch.randn(2, H, T, 2, 72, generator=gen).bfloat16().cuda()
    k, v = kv[:, :, :, 0, :64].transpose(1, 2), kv[:, :, :, 1, 8:].transpose(1, 2)
    slots = torch.randperm(blocks * bs, generator=gen)[:T].cuda()
    wide = torch.zeros(2, H, blocks, page + 32, dtype=torch.uint8, device="cuda")
    view = wide[..., 16:16 + page].transpose(1, 2)
    nrc.context_fp4_store(k, v, slots, view)
    plain = caches(nrc, 2, blocks, H, bs, fill=0)
    nrc.context_fp4_store(k.contiguous(), v.contiguous(), slots, plain)
    assert torch.equal(view, plain)
    outs = [torch.zeros_like(kv[:, :, :, 0]) for _ in range(2)]
    nrc.context_fp4_load(view, slots, *(o[..., :64].transpose(1, 2) for o in outs))
    for o, w in zip(outs, nrc.context_fp4_load(plain, slots)):
        assert torch.equal(o[..., :64].transpose(1, 2), w) and bool((o[..., 64:] == 0).all())
    # the same slots for both layers, in one list or two
    again = caches(nrc, 2, blocks, H, bs, fill=0)
    nrc.context_fp4_store(k, v, slots.expand(2, -1).contiguous(), again)
    assert torch.equal(again, plain)


def test_no_rows_graph_and_stream(nrc):
    c = caches(nrc, 2, 3, 2, 16)
    before = c.clone()
    none = torch.empty(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    nrc.context_fp4_store(none, none, slots, c)
    k, v = nrc.context_fp4_load(c, slots)
    assert torch.equal(c, before) and k.shape == none.shape and v.shape == none.shape
    kv = torch.randn(2, 9, 2, 2, 64, device="cuda").bfloat16()
    slots = torch.arange(9, device="cuda") * 5
    nrc.context_fp4_store(kv[:, :, 0], kv[:, :, 1], slots, c)
    want = c.clone()
    want_kv = nrc.context_fp4_load(c, slots)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.copy_(before)
    side.wait_stream(torch.cuda.current_stream())
    nrc.context_fp4_store(kv[:, :, 0], kv[:, :, 1], slots, c, stream=side)
    got = nrc.context_fp4_load(c, slots, stream=side)
    side.synchronize()
    assert torch.equal(c, want) and all(torch.equal(a, b) for a, b in zip(got, want_kv))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nrc.context_fp4_store(kv[:, :, 0], kv[:, :, 1], slots, c)
        held = nrc.context_fp4_load(c, slots)
    for _ in range(3):
        c.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c, want) and all(torch.equal(a, b) for a, b in zip(held, want_kv))


def test_refusals(nrc):
    c = caches(nrc, 2, 3, 2, 16)
    kv = torch.zeros(2, 9, 2, 2, 64, device="cuda", dtype=torch.bfloat16)
    k, v, slots = kv[:, :, 0], kv[:, :, 1], torch.arange(9, device="cuda")
    for bad in (dict(k=k.float()), dict(k=k.cpu()), dict(v=v[:, :8]), dict(v=v[..., ::2]), dict(slots=slots.int()),
                dict(slots=slots.cpu()), dict(slots=slots[None].expand(3, -1)), dict(slots=slots[::2]), dict(c=c.cpu()),
                dict(c=c.to(torch.int8)), dict(c=c[..., :-16]), dict(c=c[:1]), dict(c=c[0, 0]), dict(k=k[0])):
        a = dict(k=k, v=v, slots=slots, c=c)
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            nrc.context_fp4_store(a["k"], a["v"], a["slots"], a["c"])
    odd = torch.zeros(2, 9, 2, 2, 65, device="cuda", dtype=torch.bfloat16)[..., :64]
    with pytest.raises(nrc.NrcError, match="multiples of 8"):
        nrc.context_fp4_store(odd[:, :, 0], odd[:, :, 1], slots, c)
    with pytest.raises(nrc.NrcError, match="overlap"):
        nrc.context_fp4_store(k, v, slots, c[:, :, :1].expand(-1, -1, 2, -1))
    with pytest.raises(nrc.NrcError, match="overlap"):
        nrc.context_fp4_load(c, slots, k[:, :1].expand(-1, 9, -1, -1), v)
    with pytest.raises(nrc.NrcError, match="apart"):
        nrc.context_fp4_load(c, slots, k, k)
    with pytest.raises(ValueError):
        nrc.context_fp4_load(c, slots, out_k=torch.empty_like(k))
    with pytest.raises(nrc.NrcError):
        nrc.fp4_page_bytes(0)
    assert nrc.fp4_page_bytes(16) == 1088 and nrc.fp4_page_bytes(1) == 80


def test_steps_are_bf16():
    assert all(float(torch.tensor(s).bfloat16()) == s for s in STEPS)
