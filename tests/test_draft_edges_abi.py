"""Edges of the operators on a drafted token's way to the cache, without a GPU: what
the binding and the argument checks do before any launch."""

import ctypes
import os

import pytest
import torch

EINVAL = -22
at = ctypes.c_void_p


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not os.path.exists(m.library_path()):
        from norm_rope_cache_amd import build

        build.build()
    m._load()
    return m


class Recorder:
    """qk_norm_rotate_grad on the CPU: its operands' checks and its launch taken out, tensors made on the CPU."""

    def __init__(self, nrc, monkeypatch):
        self.zeros, self.calls = [], []
        monkeypatch.setattr(nrc, "_qk_operands", lambda q, k, *rest: (0, 0, ()))
        monkeypatch.setattr(nrc, "_heads", lambda t, *rest: (t.data_ptr(), *t.stride()[:2]))
        monkeypatch.setattr(nrc, "_empty", lambda shape, dtype, device, stream: torch.empty(shape, dtype=dtype))
        monkeypatch.setattr(nrc, "_stream", lambda stream, ref: stream)
        monkeypatch.setattr(nrc, "_call", lambda ref, fn, *args: self.calls.append(args))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)

        def zeros(shape, dtype, device, stream):
            self.zeros.append((tuple(shape), stream))
            return torch.zeros(shape, dtype=dtype)

        monkeypatch.setattr(nrc, "_zeros", zeros, raising=False)


def test_gradients_that_count_as_zero_are_made_on_the_calls_stream(nrc, monkeypatch):
    """Zeros of another stream would be read before they are there, and given to others while they are read."""
    rec = Recorder(nrc, monkeypatch)
    monkeypatch.setattr(torch, "zeros_like", lambda *a, **kw: pytest.fail("made on the current stream"))
    q, k = torch.randn(3, 4, 64), torch.randn(3, 2, 64)
    side = object()
    nrc.qk_norm_rotate_grad(None, k, q, k, None, None, stream=side)
    nrc.qk_norm_rotate_grad(q, None, q, k, None, None, stream=side)
    nrc.qk_norm_rotate_grad(None, None, q, None, None, None, stream=side)
    assert rec.zeros == [((3, 4, 64), side), ((3, 2, 64), side), ((3, 4, 64), side)]


def test_dual_tensors_are_refused(nrc):
    """They do not require grad: their tangents would be lost without a word."""
    import torch.autograd.forward_ad as forward

    q, k, g = torch.randn(3, 4, 64), torch.randn(3, 2, 64), torch.randn(64)
    pos, cs = torch.arange(3), torch.ones(8, 64)
    with forward.dual_level():
        dual = lambda t: forward.make_dual(t, torch.ones_like(t))
        for call in (lambda: nrc.rope_rotate(dual(q), pos, cs), lambda: nrc.rope_rotate(q, pos, dual(cs)),
                     lambda: nrc.rope_rotate(dual(q), pos, cs, out=q),
                     lambda: nrc.qk_norm_rotate(dual(q), k, pos, cs), lambda: nrc.qk_norm_rotate(q, dual(k), pos, cs),
                     lambda: nrc.qk_norm_rotate(q, k, pos, dual(cs)), lambda: nrc.qk_norm_rotate(q, k, pos, cs, dual(g), g),
                     lambda: nrc.qk_norm_rotate(q, k, pos, cs, g, dual(g)),
                     lambda: nrc.qk_norm_rotate_grad(dual(q), k, q, k, pos, cs),
                     lambda: nrc.qk_norm_rotate_grad(None, None, q, dual(k), pos, cs)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):  # (which forward mode does not heed)
                call()
        for call in (lambda: nrc.rope_rotate(q, pos, cs), lambda: nrc.qk_norm_rotate(dual(q).detach(), k, pos, cs)):
            with pytest.raises(TypeError, match="GPU"):  # no tangents: on to the other checks
                call()


def test_gains_of_no_keys(nrc, monkeypatch):
    """Keys without heads: the C entry takes no gradient of their gains, which is 0."""
    rec = Recorder(nrc, monkeypatch)
    q, k, g = torch.randn(3, 4, 64), torch.randn(3, 0, 64), torch.randn(64)
    dq, dk, dqw, dkw = nrc.qk_norm_rotate_grad(q, k, q, k, None, None, k_weight=g)
    assert dk.shape == k.shape and dqw is None and torch.equal(dkw, torch.zeros(64))
    dk_weight, ws, need = rec.calls[0][-5], rec.calls[0][-4], rec.calls[0][-3]
    assert dk_weight is None and ws is None and need == 0


Q, K, OQ, OK, POS, CS = (at(0x40000000 * i) for i in range(1, 7))  # never dereferenced


def norm_call(lib, **kw):
    ok = dict(q=Q, qr=512, qh=64, Hq=8, k=K, kr=128, kh=64, Hk=2, dtype=0, T=4, d=64, qw=None, qwt=0, kw=None, kwt=0, eps=1e-6,
              pos=POS, cs=CS, tdtype=0, maxp=10, R=64, layout=0, oq=OQ, oqr=512, oqh=64, ok=OK, okr=128, okh=64, flags=0, stream=None)
    assert not set(kw) - set(ok), kw
    return lib.nrc_qk_norm_rotate(*{**ok, **kw}.values())


def shifted(p, elements):
    return at(p.value + 2 * elements)


def view(name, p, row, head):
    return {name: p, name + "r": row, name + "h": head}


def in_place(q, k, qs, ks, **kw):
    return dict(view("q", q, *qs), **view("oq", q, *qs), **view("k", k, *ks), **view("ok", k, *ks), **kw)


def test_heads_of_one_tensor_that_meet(nrc):
    """In place over [T, H, 3, 64] and the like: what meets by an element is refused (what lies apart is launched, on a GPU)."""
    lib = nrc._load()
    by_heads = (8 * 192, 192)
    for kw in (in_place(Q, shifted(Q, 63), by_heads, by_heads, Hk=8),  # k begins in q's head
               in_place(Q, shifted(Q, 129), by_heads, by_heads, Hk=8),  # k ends in q's next head
               in_place(Q, shifted(Q, 5 * 192 + 32), by_heads, by_heads, Hk=2),
               in_place(Q, shifted(Q, 64), by_heads, (8 * 192, 160), Hk=8),  # heads that drift into each other
               in_place(Q, shifted(Q, 64), by_heads, (8 * 192 + 64, 192), Hk=8),  # rows that do
               in_place(Q, shifted(Q, 64), (192, 4 * 192), (192 - 8, 4 * 192), Hk=8),  # heads before rows
               dict(view("q", Q, *by_heads), **view("oq", shifted(Q, 32), *by_heads)),
               in_place(Q, shifted(Q, 32), (0, 192), (0, 192), T=1, Hk=8), in_place(Q, shifted(Q, 32), (64, 0), (64, 0), Hq=1, Hk=1)):
        assert norm_call(lib, **kw) == EINVAL and b"apart" in lib.nrc_last_error(), kw


def test_loaded_rows_of_one_tensor_that_meet(nrc):
    """K and V by turns in one tensor: what meets by a few elements is refused."""
    lib = nrc._load()

    def call(v, ks, vs, T=4, H=2, L=3):
        return lib.nrc_context_fp4_load(at(0x10000), 1 << 20, 2176, 1088, 8, 16, POS, 0, T, H, L, K, *ks, v, *vs, 0, None)

    rows = (4 * 256, 256, 64)  # [3, 4, 2 (K, V), 2, 64]
    for v, ks, vs, kw in ((shifted(K, 120), rows, rows, {}), (shifted(K, 136), rows, rows, {}),
                          (shifted(K, 128), rows, (4 * 256, 264, 64), {}), (shifted(K, 128), rows, (4 * 256 + 8, 256, 64), {}),
                          (shifted(K, 72), (2048, 256, 128), (2048, 256, 128), {}),
                          (shifted(K, 56), (2048, 256, 128), (2048, 256, 128), dict(T=1, L=1))):
        assert call(v, ks, vs, **kw) == EINVAL and b"apart" in lib.nrc_last_error(), (v, ks, vs)


def test_reference_of_all_rows_at_once(monkeypatch):
    """dense_attention against the row by row reference, with a window, sinks and a block that is not there."""
    import cache_ref
    from draft_ref import dense_attention, make_batch

    to = torch.Tensor.to
    monkeypatch.setattr(torch.Tensor, "to", lambda t, *a, **kw: t if a[:1] == ("cuda",) else to(t, *a, **kw))
    for f in ("zeros", "full", "arange"):
        made = getattr(torch, f)
        monkeypatch.setattr(torch, f, lambda *a, made=made, **kw: made(*a, **{k: v for k, v in kw.items() if k != "device"}))
    for window in (None, 11):
        bt = make_batch()([40, 0, 17], [5, 3, 2], H=2, G=3, block_size=4, tree=False, seed=2).behind(window, 3)
        bt.tables[0, 7] = -1
        bt.tables[2, :] = bt.nb  # nothing at all
        for a, b in zip(dense_attention(bt), cache_ref.attention(bt)):
            assert torch.allclose(a, b, rtol=1e-9, atol=1e-12)


def gains_inputs(T, heads, d, along, seed):
    """x, its outputs' gradients, gains, positions and a table; along: gradients that are near the outputs, so that the gains' sums
    grow with every row."""
    from draft_ref import turn

    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, heads, d, generator=gen).bfloat16()
    w = 1 + 0.2 * torch.randn(d, generator=gen)
    pos = torch.randint(0, 300, (T,), generator=gen)
    angle = torch.arange(300)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d / 2))
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    g = torch.randn(T, heads, d, generator=gen)
    if along:
        g = turn(x.double(), pos, cs, "half")[0].float() + 0.1 * g
    return x, g.bfloat16(), w, pos, cs


@pytest.mark.parametrize("along", [False, True])
def test_bound_of_the_gains_gradients_rejects_lost_rows(along):
    """Of 4099 rows of 23 heads: one row, a workgroup's rows, the last of a walk's rounds left out, heads counted twice, all of it
    lost; and the sums in FP32 in another order are within it."""
    from draft_ref import gains_grad, sum_depth

    x, g, w, pos, cs = gains_inputs(4099, 23, 64, along, 5)
    depth = sum_depth(4099, 23, 3, 4, 256)
    assert depth < 128
    dw, tol = gains_grad(g, x, w, pos, cs, "half", 1e-6, depth)
    rejects = lambda other: int(((other - dw).abs() > tol).sum())
    part = lambda rows: gains_grad(g[rows], x[rows], w, pos[rows], cs, "half", 1e-6, depth)[0]
    one = part(slice(4098, 4099))
    assert rejects(dw - one) >= 50 and rejects(dw + one) >= 50
    for rows in (slice(100, 106), slice(4000, 4099), slice(0, 2)):
        assert rejects(dw - part(rows)) >= 50, rows
    assert rejects(torch.zeros_like(dw)) == 64
    xf, gf = x.float(), g.float()
    u = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6)
    back = cs[pos][:, None, :]
    a, b = gf[..., :32], gf[..., 32:]
    gf = torch.cat([a * back[..., :32] + b * back[..., 32:], b * back[..., :32] - a * back[..., 32:]], -1)
    assert rejects((gf * u).flip(0).sum((0, 1)).double()) == 0
