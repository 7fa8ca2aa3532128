"""The operators on a drafted token's way to the cache, without a GPU: bad
arguments are refused on the host before any launch, empty calls touch nothing;
the references' own checks."""

import ctypes
import math
import os

import pytest
import torch

import cache_ref
from draft_ref import STEPS, fp4_groups, fp4_values, make_batch, norm_rotate, norm_rotate_grad

EINVAL, ENOTSUP = -22, -95
at = ctypes.c_void_p
FAKE = at(0x10000)  # aligned non-NULL addresses that are never dereferenced, far from each other
Q, K, OQ, OK, W, POS, CS, WS = (at(0x40000000 * i) for i in range(1, 9))
MISALIGNED = at(0x10001)


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


HEADS = dict(q=Q, qr=512, qh=64, Hq=8, k=K, kr=128, kh=64, Hk=2, dtype=0, T=4, d=64, qw=None, qwt=0, kw=None, kwt=0, eps=1e-6,
             pos=POS, cs=CS, tdtype=0, maxp=10, R=64, layout=0)
QK_NOTSUP = [dict(dtype=3), dict(dtype=-1), dict(tdtype=1), dict(d=257), dict(d=1), dict(T=(1 << 25) + 1), dict(Hq=1 << 24),
             dict(qw=W, qwt=3), dict(kw=W, kwt=-1)]
QK_EINVAL = [dict(layout=2), dict(T=-1), dict(Hq=0), dict(Hk=-1), dict(R=0), dict(R=3), dict(R=66), dict(maxp=0), dict(maxp=1 << 29),
             dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(pos=None), dict(cs=None), dict(q=None), dict(k=None),
             dict(q=MISALIGNED), dict(pos=at(0x10004)), dict(tdtype=2, cs=at(0x10002)), dict(qw=MISALIGNED),
             dict(kw=at(0x10002), kwt=2), dict(qr=-1), dict(kh=1 << 41)]


def test_qk_norm_rotate(lib):
    call = caller(lib.nrc_qk_norm_rotate, dict(HEADS, oq=OQ, oqr=512, oqh=64, ok=OK, okr=128, okh=64, flags=0, stream=None))
    for kw in QK_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    for kw in QK_EINVAL + [dict(flags=2), dict(oq=None), dict(ok=None), dict(oqh=63), dict(oqr=511), dict(okr=0)]:
        assert call(**kw) == EINVAL, kw
        assert b"qk_norm_rotate" in lib.nrc_last_error()
    # an output over another operand, another strided view of its input, the other output
    for kw in (dict(oq=K), dict(ok=Q), dict(oq=OK), dict(oq=Q, oqr=1024), dict(oq=at(Q.value + 2)), dict(oq=POS), dict(ok=CS),
               dict(qw=OQ), dict(kw=OQ, oqr=600), dict(oq=at(Q.value + 64 * 2 * 8 * 3))):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    # parts of one wider row that overlap by an element, and a k that begins inside q
    row = dict(qr=704, kr=704, oqr=704, okr=704, oq=Q)
    for k in (at(Q.value + 511 * 2), at(Q.value + 2 * 2 * 704 + 511 * 2), at(Q.value + 2 * (704 - 127))):
        assert call(**row, k=k, ok=k) == EINVAL and b"apart" in lib.nrc_last_error()
    assert call(T=0, q=None, k=None, pos=None, cs=None, oq=None, ok=None) == 0
    assert call(T=0, Hk=0, k=None, ok=None) == 0


def test_qk_norm_rotate_grad(lib):
    ok = dict(gq=at(Q.value + 0x1000000), gqr=512, gqh=64, gk=at(K.value + 0x1000000), gkr=128, gkh=64, **HEADS, dq=OQ, dk=OK,
              dqw=None, dkw=None, ws=None, bytes=0, flags=0, stream=None)
    call = caller(lib.nrc_qk_norm_rotate_grad, ok)
    need = lib.nrc_qk_norm_rotate_grad_workspace_bytes(64, 1)
    assert need > 0 and lib.nrc_qk_norm_rotate_grad_workspace_bytes(64, 0) == 0
    assert lib.nrc_qk_norm_rotate_grad_workspace_bytes(257, 1) == ENOTSUP
    for kw in QK_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    gains = dict(qw=W, dqw=at(W.value + 0x1000), ws=WS, bytes=need)
    for kw in QK_EINVAL + [dict(flags=2), dict(dq=None), dict(dk=None), dict(gq=None), dict(gk=None), dict(gkr=-8),
                           dict(gains, dqw=None), dict(dqw=W), dict(dkw=W), dict(gains, bytes=need - 1), dict(gains, ws=None),
                           dict(gains, ws=at(WS.value + 8)), dict(gains, qwt=2, dqw=at(W.value + 0x1002))]:
        assert call(**kw) == EINVAL, kw
        assert b"qk_norm_rotate_grad" in lib.nrc_last_error()
    for kw in (dict(dq=Q), dict(dq=K), dict(dk=OQ), dict(dq=at(Q.value + 0x1000000)), dict(gains, dqw=W), dict(gains, ws=Q),
               dict(gains, ws=OQ), dict(gains, dqw=POS), dict(gains, ws=W), dict(dk=CS)):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    assert call(T=0, q=None, k=None, pos=None, cs=None, gq=None, gk=None, dq=None, dk=None) == 0


PAGES = dict(c=FAKE, ls=1 << 20, bst=2176, hst=1088, nb=8, bs=16)
ROWS = dict(k=K, kl=4096, kr=128, kh=64, v=Q, vl=4096, vr=128, vh=64)
PAGES_NOTSUP = [dict(ls=8), dict(bst=2184), dict(hst=1089), dict(nb=1 << 27), dict(nb=1, bs=(1 << 24) + 1), dict(H=65536)]
PAGES_EINVAL = [dict(nb=0), dict(bs=0), dict(H=0), dict(bst=-16), dict(hst=1 << 41), dict(c=None), dict(c=at(0x10008))]
ROWS_EINVAL = [dict(T=-1), dict(L=-1), dict(k=None), dict(v=None), dict(k=at(0x10008)), dict(kl=4), dict(kr=-8), dict(vh=1 << 41),
               dict(slots=None), dict(slots=at(0x10004)), dict(sl=-1)]


def test_fp4_page_bytes(lib):
    for bs in range(1, 300):
        n = lib.nrc_fp4_page_bytes(bs)
        assert n % 16 == 0 and 68 * bs <= n < 68 * bs + 16
    assert lib.nrc_fp4_page_bytes(0) == EINVAL and lib.nrc_fp4_page_bytes((1 << 24) + 1) == EINVAL


def test_fp4_store(lib):
    call = caller(lib.nrc_context_fp4_store, dict(ROWS, slots=POS, sl=0, T=4, H=2, L=3, **PAGES, stream=None))
    for kw in PAGES_NOTSUP + [dict(T=(1 << 28) + 1), dict(L=65536)]:
        assert call(**kw) == ENOTSUP, kw
    for kw in PAGES_EINVAL + ROWS_EINVAL:
        assert call(**kw) == EINVAL, kw
        assert b"context_fp4_store" in lib.nrc_last_error()
    for kw in (dict(bst=1088), dict(hst=0), dict(ls=0), dict(ls=2176), dict(hst=1072)):
        assert call(**kw) == EINVAL and b"overlap" in lib.nrc_last_error(), kw
    for kw in (dict(c=K), dict(c=at(Q.value + 4096 * 2 * 2)), dict(c=POS), dict(c=at(POS.value - 1088 - 7 * 2176 - 2 * (1 << 20)))):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    assert call(T=0, k=None, v=None, slots=None, c=None) == 0 and call(L=0, k=None, v=None, slots=None, c=None) == 0


def test_fp4_load(lib):
    call = caller(lib.nrc_context_fp4_load, dict(PAGES, slots=POS, sl=0, T=4, H=2, L=3, **ROWS, flags=0, stream=None))
    for kw in PAGES_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    for kw in PAGES_EINVAL + ROWS_EINVAL + [dict(flags=2)]:
        assert call(**kw) == EINVAL, kw
        assert b"context_fp4_load" in lib.nrc_last_error()
    for kw in (dict(kr=64), dict(kh=56), dict(kl=0), dict(vl=256)):
        assert call(**kw) == EINVAL and b"overlap" in lib.nrc_last_error(), kw
    for kw in (dict(k=Q), dict(v=FAKE), dict(k=POS), dict(k=at(Q.value + 4096 * 2))):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    assert call(T=0, k=None, v=None, slots=None, c=None) == 0


TABLES = dict(tables=FAKE, ts=4, tw=4, B=3)
QUERIES = dict(q=Q, qr=512, qh=64, T=6, Hq=8)
REST = dict(ctx=FAKE, starts=FAKE, nodes=2, max_ctx=60, mask=None, words=0, scale=0.125, cap=0.0, window=8, sinks=2, out=OQ, lse=OK,
            ws=None, ws_bytes=0, flags=0, stream=None)
QUERY_NOTSUP = [dict(Hq=7), dict(T=1 << 31), dict(B=60000, nodes=60000), dict(scale=1e-13), dict(cap=1025.0), dict(B=65536)]
QUERY_EINVAL = [dict(T=-1), dict(nodes=0), dict(nodes=65536), dict(max_ctx=-1), dict(max_ctx=1 << 31), dict(qr=4), dict(words=1),
                dict(mask=FAKE), dict(mask=FAKE, words=1, nodes=65), dict(scale=0.0), dict(scale=math.nan), dict(cap=-1.0),
                dict(q=None), dict(ctx=None), dict(starts=None), dict(q=at(0x10008)), dict(tw=0), dict(ts=-1), dict(tables=None),
                dict(tables=at(0x10002)), dict(window=-1), dict(sinks=-1), dict(flags=4), dict(out=None), dict(lse=None),
                dict(out=at(0x10008)), dict(lse=at(0x10002))]


def check_attention(lib, call, name, cache):
    for kw in QUERY_NOTSUP:
        assert call(**kw) == ENOTSUP, kw
    for kw in QUERY_EINVAL:
        assert call(**kw) == EINVAL, kw
        assert name in lib.nrc_last_error()
    for kw in (dict(out=Q), dict(lse=Q), dict(lse=OQ), dict(out=cache), dict(lse=cache), dict(out=FAKE), dict(lse=FAKE)):
        assert call(**kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw
    long = dict(max_ctx=200000, B=1, tw=20000, window=150000, nodes=6)
    need = lib.nrc_context_window_attention_workspace_bytes(1, 6, 8, 2, 6, 200000, 150000, 2)
    assert need > 0
    for kw in (dict(), dict(ws=WS, ws_bytes=need - 1), dict(ws=at(WS.value + 8), ws_bytes=need)):
        assert call(**long, **kw) == EINVAL and b"workspace" in lib.nrc_last_error(), kw
    for ws in (Q, OQ, OK, cache):
        assert call(**long, ws=ws, ws_bytes=need) == EINVAL and b"apart" in lib.nrc_last_error()
    nothing = dict(q=None, tables=None, ctx=None, starts=None, out=None, lse=None)
    assert call(**nothing, B=0) == 0 and call(**nothing, T=0) == 0


def test_window_attention(lib):
    paged = dict(c=K, nb=8, bs=16, bst=2 * 16 * 128, pst=128, hst=16 * 128, H=2)
    call = caller(lib.nrc_context_window_attention, dict(QUERIES, **paged, **TABLES, **REST))
    check_attention(lib, call, b"context_window_attention", K)
    for kw in (dict(nb=1 << 27), dict(bst=4), dict(pst=132)):
        assert call(**kw) == ENOTSUP, kw
    for kw in (dict(window=0), dict(c=None), dict(c=at(0x10008)), dict(nb=0)):
        assert call(**kw) == EINVAL, kw


def test_fp4_attention(lib):
    paged = dict(c=K, nb=8, bs=16, bst=2176, hst=1088, H=2)
    call = caller(lib.nrc_context_fp4_attention, dict(QUERIES, **paged, **TABLES, **REST))
    check_attention(lib, call, b"context_fp4_attention", K)
    for kw in (dict(nb=1 << 27), dict(bst=2184), dict(hst=8)):
        assert call(**kw) == ENOTSUP, kw
    for kw in (dict(c=None), dict(c=at(0x10008)), dict(nb=0), dict(bs=0)):
        assert call(**kw) == EINVAL, kw


def test_attention_workspace(lib):
    f = lib.nrc_context_window_attention_workspace_bytes
    assert f(0, 6, 8, 2, 2, 100000, 10, 0) == 0 and f(1, 0, 8, 2, 2, 100000, 10, 0) == 0
    assert f(1, 6, 8, 2, 2, 1 << 20, 64, 4) == 0  # a short window over a long context
    assert f(1, 6, 8, 2, 2, 1 << 20, 0, 0) > 0 and f(1, 600, 8, 2, 600, 1 << 20, 0, 0) > 0
    assert f(1, 6, 8, 2, 2, 100, -1, 0) == EINVAL and f(1, 6, 8, 2, 2, 100, 1, -1) == EINVAL
    assert f(1, 6, 7, 2, 2, 100, 1, 0) == ENOTSUP
    # bounded, whatever the sizes: the partial sums of what the chip holds a few times over
    for B in (1, 7, 64, 512, 4096):
        for H, G in ((1, 1), (8, 8), (64, 2)):
            for nodes in (1, 3, 40, 500):
                for window in (0, 1000, 2 ** 31 - 1):
                    n = f(B, B * nodes, H * G, H, nodes, 1 << 20, window, 4)
                    assert n < 1 << 28 or n == ENOTSUP, (B, H, G, nodes, window, n)


# ---- the references' own checks -----------------------------------------------------------------------------------

def test_reference_of_the_cells():
    """Values by hand: scales at the borders, ties to the even code, the held exponents."""
    row = torch.zeros(64, dtype=torch.float64)
    row[:8] = torch.tensor([6.0, 5.0, 2.5, 3.5, 1.25, 0.25, -0.75, -1.75])
    row[32:36] = torch.tensor([6.25, 1.0, 0.5, -3.0])
    want = torch.zeros_like(row)
    want[:8] = torch.tensor([6.0, 4.0, 2.0, 4.0, 1.0, 0.0, -1.0, -2.0])
    want[32:36] = torch.tensor([6.0, 1.0, 0.0, -3.0])  # scale 2: 3.125 -> 3, 0.5 -> 0.5, 0.25 -> 0, -1.5
    assert torch.equal(fp4_values(row), want)
    for v, e in ((6 * 2.0 ** 125, 125), (2.0 ** 127 * 1.9, 125), (3.0, -1), (3.0001, 0), (2.0 ** -130, -120), (0.0, -120)):
        g = torch.zeros(32, dtype=torch.float64)
        g[3] = v
        assert int(fp4_groups(g)[1]) == e, v
    assert STEPS == sorted(STEPS)


def test_reference_of_the_norm():
    """The formula's gradient against torch's differentiation of the forward reference."""
    gen = torch.Generator().manual_seed(1)
    for layout in ("interleaved", "half"):
        x = torch.randn(5, 3, 64, generator=gen).double().requires_grad_()
        w = torch.randn(64, generator=gen).double().requires_grad_()
        g = torch.randn(5, 3, 64, generator=gen).double()
        pos = torch.randint(0, 20, (5,), generator=gen)
        a = torch.arange(20)[:, None] * 100.0 ** (-torch.arange(16) / 16)
        cs = torch.cat([a.cos(), a.sin()], 1)
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
        y = n.clone()
        row = cs.double()[pos][:, None, :]
        ia, ib = (slice(0, 32, 2), slice(1, 32, 2)) if layout == "interleaved" else (slice(0, 16), slice(16, 32))
        y = torch.cat([torch.stack([n[..., ia] * row[..., :16] - n[..., ib] * row[..., 16:],
                                    n[..., ib] * row[..., :16] + n[..., ia] * row[..., 16:]], -1).flatten(-2) if layout == "interleaved"
                       else torch.cat([n[..., ia] * row[..., :16] - n[..., ib] * row[..., 16:],
                                       n[..., ib] * row[..., :16] + n[..., ia] * row[..., 16:]], -1), n[..., 32:]], -1)
        assert torch.allclose(norm_rotate(x.detach(), w.detach(), pos, cs, layout, 1e-5)[0], y.detach(), rtol=1e-12, atol=1e-14)
        dx, dw = torch.autograd.grad(y, (x, w), g)
        rx, _, rw, _ = norm_rotate_grad(g, x.detach(), w.detach(), pos, cs, layout, 1e-5)
        assert torch.allclose(rx, dx, rtol=1e-10, atol=1e-12) and torch.allclose(rw, dw, rtol=1e-10, atol=1e-12)


def test_reference_of_the_window():
    """Which keys a chain's and a tree's rows see, by hand."""
    Batch = make_batch()
    bt = Batch([6], [3], H=1, G=1, tree=False).behind(4, 2)
    there = torch.ones(9, dtype=torch.bool).numpy()
    want = [[0, 1, 3, 4, 5, 6], [0, 1, 4, 5, 6, 7], [0, 1, 5, 6, 7, 8]]
    assert [r.nonzero().flatten().tolist() for r in bt.sees(0, there)] == want
    bt = Batch([6], [3], H=1, G=1, tree=True).behind(2, 1)
    bt.mask = cache_ref.tree_words([-1, 0, 0], 1)  # two children of one root: depth 1 both
    want = [[0, 5, 6], [0, 6, 7], [0, 6, 8]]  # positions 6, 7, 7; of the context the sinks and key 5 alone
    assert [r.nonzero().flatten().tolist() for r in bt.sees(0, there)] == want
