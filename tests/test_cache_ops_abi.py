"""The operators around the cache without a GPU: bad arguments are refused on
the host before any launch, empty calls touch nothing; the references' own
checks."""

import ctypes
import math
import os

import pytest

EINVAL, ENOTSUP = -22, -95
FAKE = ctypes.c_void_p(0x10000)  # an aligned non-NULL address that is never dereferenced
FAR = ctypes.c_void_p(0x40000000)
MISALIGNED = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    import norm_rope_cache_amd as m

    if not os.path.exists(m.library_path()):
        from norm_rope_cache_amd import build

        build.build()
    return m._load()


def caller(f, ok):
    def call(**kw):
        assert not set(kw) - set(ok), kw
        return f(*{**ok, **kw}.values())

    return call


def test_rope_table(lib):
    call = caller(lib.nrc_rope_table, dict(start=0, count=8, R=64, width=64, base=1e4, scaling=0, factor=1.0, orig=1.0,
                                           low=1.0, high=2.0, magnitude=1.0, out=FAKE, dtype=0, stream=None))
    for kw in (dict(dtype=1), dict(dtype=3), dict(R=0), dict(R=3), dict(R=258, width=258)):
        assert call(**kw) == ENOTSUP, kw
    for kw in (dict(width=62), dict(width=65), dict(width=514), dict(scaling=-1), dict(scaling=5),
               dict(magnitude=math.nan), dict(start=-1), dict(count=-1), dict(start=1 << 28), dict(count=(1 << 28) + 1),
               dict(start=2 ** 63 - 1, count=2 ** 63 - 1), dict(base=1.0), dict(base=math.inf), dict(base=math.nan),
               dict(scaling=1, factor=0.0), dict(scaling=1, factor=math.nan), dict(scaling=2, R=2, factor=2.0),
               dict(scaling=3, orig=0.0), dict(scaling=4, low=0.0), dict(scaling=4, high=1.0), dict(out=None),
               dict(out=MISALIGNED, dtype=2)):
        assert call(**kw) == EINVAL, kw
        assert b"rope_table" in lib.nrc_last_error()
    assert call(count=0, out=None) == 0


def test_rope_rotate(lib):
    call = caller(lib.nrc_rope_rotate, dict(x=FAKE, dtype=0, T=4, H=2, d=64, xr=128, xh=64, pos=FAKE, cs=FAKE, tdtype=0,
                                            maxp=10, R=64, layout=0, inverse=0, out=FAR, orr=128, oh=64, stream=None))
    for kw in (dict(dtype=3), dict(dtype=-1), dict(tdtype=1), dict(T=(1 << 23) + 1), dict(H=2000)):
        assert call(**kw) == ENOTSUP, kw
    for kw in (dict(layout=2), dict(inverse=2), dict(T=-1), dict(H=0), dict(d=0), dict(R=0), dict(R=3), dict(R=66),
               dict(maxp=0), dict(maxp=1 << 29), dict(x=None), dict(pos=None), dict(cs=None), dict(out=None),
               dict(x=ctypes.c_void_p(0x10001)), dict(dtype=2, x=MISALIGNED), dict(pos=MISALIGNED),
               dict(tdtype=2, cs=MISALIGNED), dict(xr=-1), dict(oh=1 << 41), dict(oh=63), dict(orr=127), dict(orr=0),
               dict(out=FAKE, orr=256), dict(out=ctypes.c_void_p(FAKE.value + 1022))):
        assert call(**kw) == EINVAL, kw
    assert call(T=0, x=None, pos=None, cs=None, out=None) == 0


PAGED = dict(cache=FAKE, nb=8, bs=16, bst=2 * 16 * 128, pst=128, hst=16 * 128, H=2, tables=FAKE, ts=4, tw=4, B=3)
QUERIES = dict(q=FAKE, qr=512, qh=64, T=6, Hq=8, **PAGED, ctx=FAKE, starts=FAKE, nodes=2, max_ctx=60, mask=None, words=0,
               scale=0.125, cap=0.0)
PAGED_NOTSUP = [dict(nb=1 << 27), dict(bst=4), dict(pst=132), dict(hst=1), dict(H=65536, Hq=65536), dict(B=65536)]
PAGED_EINVAL = [dict(H=0), dict(B=-1), dict(nb=0), dict(bs=0), dict(bst=-8), dict(pst=-8), dict(hst=1 << 41), dict(tw=0),
                dict(tw=1 << 40), dict(ts=-1), dict(cache=None), dict(tables=None), dict(cache=ctypes.c_void_p(0x10008)),
                dict(tables=MISALIGNED)]
QUERY_NOTSUP = [dict(Hq=7), dict(T=1 << 31), dict(B=60000, nodes=60000), dict(scale=1e-13), dict(scale=2e12),
                dict(cap=9e-4), dict(cap=1025.0)]
QUERY_EINVAL = [dict(T=-1), dict(Hq=0), dict(nodes=0), dict(nodes=65536), dict(max_ctx=-1), dict(max_ctx=1 << 31), dict(qr=4),
                dict(qh=-8), dict(words=1), dict(mask=FAKE), dict(mask=FAKE, words=-1), dict(mask=FAKE, words=1, nodes=65),
                dict(mask=MISALIGNED, words=1), dict(mask=FAKE, words=1025), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.nan), dict(q=None),
                dict(ctx=None), dict(starts=None), dict(q=ctypes.c_void_p(0x10008)), dict(ctx=MISALIGNED),
                dict(starts=MISALIGNED)]


def test_tree_attention(lib):
    call = caller(lib.nrc_context_tree_attention, dict(QUERIES, out=FAR, lse=ctypes.c_void_p(0x20000000), ws=None,
                                                       ws_bytes=0, stream=None))
    for kw in PAGED_NOTSUP + QUERY_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    for kw in PAGED_EINVAL + QUERY_EINVAL + [dict(out=None), dict(lse=None), dict(out=ctypes.c_void_p(0x10008)),
                                             dict(lse=MISALIGNED)]:
        assert call(**kw) == EINVAL, kw
        assert b"context_tree_attention" in lib.nrc_last_error()
    for kw in (dict(out=FAKE), dict(lse=FAKE), dict(out=ctypes.c_void_p(FAKE.value + 2 * (5 * 512 + 7 * 64 + 56))),
               dict(lse=ctypes.c_void_p(FAR.value + 6 * 8 * 64 * 2 - 4))):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    # a long context needs a workspace
    long = dict(max_ctx=100000, B=1, tw=10000)
    need = lib.nrc_context_tree_attention_workspace_bytes(1, 6, 8, 2, 2, 100000)
    assert need > 0
    assert call(**long) == EINVAL
    assert call(**long, ws=FAKE, ws_bytes=need - 1) == EINVAL
    assert call(**long, ws=ctypes.c_void_p(0x10008), ws_bytes=need) == EINVAL
    # nothing to do
    assert call(B=0, cache=None, tables=None, q=None, ctx=None, starts=None, out=None, lse=None) == 0
    assert call(T=0, cache=None, tables=None, q=None, out=None, lse=None) == 0


def test_tree_attention_workspace(lib):
    f = lib.nrc_context_tree_attention_workspace_bytes
    assert f(0, 6, 8, 2, 2, 100000) == 0 and f(1, 0, 8, 2, 2, 100000) == 0
    assert f(1, 6, 8, 2, 2, 30) == 0  # one split
    assert f(1, 6, 7, 2, 2, 30) == ENOTSUP and f(1, 6, 8, 2, 0, 30) == EINVAL and f(1, 6, 8, 0, 2, 30) == EINVAL
    # partial sums (64 and two statistics) of every row in whole splits
    assert f(1, 6, 8, 2, 2, 100000) % (6 * 8 * 66 * 4) == 0


def test_attention_mass(lib):
    call = caller(lib.nrc_context_attention_mass, dict(QUERIES, lse=FAKE, w=FAKE, wb=200, wh=100, decay=1.0, out=FAR, ob=200,
                                                       oh=100, width=64, stream=None))
    for kw in PAGED_NOTSUP + QUERY_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    for kw in PAGED_EINVAL + QUERY_EINVAL + [dict(lse=None), dict(out=None), dict(w=MISALIGNED), dict(out=MISALIGNED),
                                             dict(lse=MISALIGNED), dict(wb=-1), dict(oh=-1), dict(width=-1),
                                             dict(width=1 << 31), dict(decay=math.inf), dict(oh=63), dict(ob=100),
                                             dict(w=FAR, wh=101), dict(w=ctypes.c_void_p(FAR.value + 4)),
                                             dict(w=ctypes.c_void_p(FAR.value + 4 * 563))]:
        assert call(**kw) == EINVAL, kw
        assert b"context_attention_mass" in lib.nrc_last_error()
    assert call(B=0, cache=None, tables=None, q=None, ctx=None, starts=None, lse=None, out=None) == 0
    assert call(width=0, cache=None, tables=None, lse=None, out=None) == 0


def test_kv_evict(lib):
    call = caller(lib.nrc_context_kv_evict, dict(PAGED, lens=FAKE, w=FAKE, wb=128, wh=64, p=FAKE, pb=128, ph=64, width=64,
                                                 ends=FAKE, sinks=0, recent=0, budget=40, nw=FAKE, np=FAKE, nl=FAKE,
                                                 ws=None, ws_bytes=0, stream=None))
    for kw in [dict(nb=1 << 27), dict(bst=4), dict(pst=132), dict(hst=1), dict(H=65535)]:
        assert call(**kw, **({"ws": FAKE, "ws_bytes": 1 << 40})) == ENOTSUP, kw
    for kw in PAGED_EINVAL + [dict(budget=0), dict(budget=-1), dict(sinks=-1), dict(recent=-1), dict(width=-1),
                              dict(width=1 << 31), dict(w=None), dict(p=None), dict(w=MISALIGNED), dict(p=MISALIGNED),
                              dict(wb=-1), dict(ph=1 << 41), dict(nw=None), dict(np=None), dict(nl=None), dict(lens=None),
                              dict(ends=None), dict(nw=MISALIGNED), dict(np=MISALIGNED), dict(nl=MISALIGNED),
                              dict(lens=MISALIGNED), dict(ends=MISALIGNED)]:
        assert call(**kw, **({"ws": FAKE, "ws_bytes": 1 << 40} if "ws" not in kw else {})) == EINVAL, kw
    # what is written lies apart from what is read
    at = [ctypes.c_void_p(0x100000 * i) for i in range(1, 8)]
    apart = dict(lens=at[0], w=at[1], p=at[2], ends=at[3], nw=at[4], np=at[5], nl=at[6])
    for out, size in (("nw", 3 * 2 * 40), ("np", 3 * 2 * 40), ("nl", 3)):
        for name, cells in (("w", 2 * 128 + 64 + 64), ("p", 2 * 128 + 64 + 64), ("lens", 3), ("ends", 3)):
            for place in (apart[name].value + 4 * (cells - 1), apart[name].value, apart[name].value - 4 * (size - 1)):
                kw = dict(apart, **{out: ctypes.c_void_p(place)})
                assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), (out, name, hex(place))
    long = dict(width=20000, wb=40000, wh=20000, pb=40000, ph=20000, budget=5000, tw=2000)
    need = lib.nrc_context_kv_evict_workspace_bytes(3, 2, 20000, 5000)
    assert need >= 2 * 6 * 5000 * 4  # two lists of as many cells as can move
    assert call(**long) == EINVAL and call(**long, ws=FAKE, ws_bytes=need - 1) == EINVAL
    assert call(**long, ws=ctypes.c_void_p(0x10008), ws_bytes=need) == EINVAL
    assert call(B=0, cache=None, tables=None, lens=None, w=None, p=None, nw=None, np=None, nl=None, ends=None) == 0
    f = lib.nrc_context_kv_evict_workspace_bytes
    assert f(3, 2, 64, 64) == 0 and f(3, 2, 64, 100) == 0 and f(0, 2, 64, 4) == 0
    assert f(3, 2, -1, 4) == EINVAL and f(3, 0, 64, 4) == EINVAL and f(3, 2, 64, 0) == EINVAL


def test_host_tensors_are_refused():
    """The binding hands no host pointer to a kernel."""
    torch = pytest.importorskip("torch")
    import norm_rope_cache_amd as nrc

    cache = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    i = lambda *shape: torch.zeros(*shape, dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        nrc.context_tree_attention(q, cache, i(1, 4), i(1), i(2), 3)
    with pytest.raises(TypeError):
        nrc.context_attention_mass(q, cache, i(1, 4), i(1), i(2), torch.zeros(3, 4), 3)
    with pytest.raises(TypeError):
        nrc.context_kv_evict(cache, i(1, 4), i(1), torch.zeros(1, 2, 64), i(1, 2, 64), i(1), 10)
    with pytest.raises(TypeError):
        nrc.rope_rotate(q, torch.zeros(3, dtype=torch.int64), torch.zeros(5, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        nrc.rope_table(4, 64, device="cpu")


def test_references():
    """The references against torch's softmax over a gathered cache, and a cell-by-cell eviction."""
    torch = pytest.importorskip("torch")
    import cache_ref as ref

    bt = ref.Batch([40], [5], H=2, G=2, tree=False)
    out, lse, _, _ = ref.attention(bt)
    k, v, there = bt.keys(0, 1, 45)
    s = bt.q[:, 3].double() @ k.T / 8
    s = s.masked_fill(~torch.tril(torch.ones(45, 45, dtype=torch.bool))[40:], -math.inf)
    assert torch.allclose(out[:, 3], torch.softmax(s, -1) @ v, atol=1e-12)
    assert torch.allclose(lse[:, 3], torch.logsumexp(s, -1), atol=1e-12)
    m, _ = ref.mass(bt, lse.float(), 45)
    assert torch.allclose(m.sum(-1), torch.full((1, 2), 10.0, dtype=torch.float64), atol=1e-5)
    c = ref.Batch([6], [0], H=1, G=1, block_size=2, tree=False)
    w = torch.tensor([[[3.0, 1.0, 5.0, 1.0, 4.0, 2.0]]])
    p = torch.arange(6, dtype=torch.int32).view(1, 1, 6)
    nw, npos, nl, cache = ref.evict(c.cache, c.tables, c.ctx_lens, w, p, c.ctx_lens, 4, 0, 0)
    assert nw.flatten().tolist() == [3.0, 4.0, 5.0, 2.0] and npos.flatten().tolist() == [0, 4, 2, 5]
    cells = lambda t, j: t[int(c.tables[0, j // 2]), 0, j % 2]
    assert torch.equal(cells(cache, 1), cells(c.cache, 4)) and torch.equal(cells(cache, 3), cells(c.cache, 5))
    assert torch.equal(cells(cache, 2), cells(c.cache, 2))
