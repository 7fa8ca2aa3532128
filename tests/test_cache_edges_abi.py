"""Calls of the operators around the cache that are refused on the host (no GPU)."""

import ctypes
import math

import pytest

from test_cache_ops_abi import EINVAL, ENOTSUP, FAKE, FAR, QUERIES, caller, lib  # noqa: F401


def test_rope_rotate_flags(lib):
    call = caller(lib.nrc_rope_rotate_ex, dict(x=FAKE, dtype=0, T=4, H=2, d=64, xr=128, xh=64, pos=FAKE, cs=FAKE, tdtype=0,
                                               maxp=10, R=64, layout=0, inverse=0, out=FAR, orr=128, oh=64, flags=1,
                                               stream=None))
    for flags in (2, 3, 1 << 31):
        assert call(flags=flags) == EINVAL and b"flags" in lib.nrc_last_error()
    assert call(layout=2) == EINVAL and call(dtype=3) == ENOTSUP
    assert call(T=0, x=None, pos=None, cs=None, out=None) == 0


def test_tree_attention_flags(lib):
    call = caller(lib.nrc_context_tree_attention_ex, dict(QUERIES, out=FAR, lse=ctypes.c_void_p(0x20000000), ws=None,
                                                          ws_bytes=0, flags=3, stream=None))
    for flags in (4, 7, 1 << 31):
        assert call(flags=flags) == EINVAL and b"flags" in lib.nrc_last_error()
    assert call(Hq=7) == ENOTSUP and call(q=None) == EINVAL and call(out=FAKE) == EINVAL
    assert call(B=0, out=None) == EINVAL and call(B=0, lse=None) == EINVAL  # every row is to be written
    assert call(T=0, q=None, cache=None, tables=None, out=None, lse=None) == 0


def at(p, offset):
    return ctypes.c_void_p(p.value + offset)


def test_rope_rotate_out_apart_from_what_it_reads(lib):
    """Positions of 4 rows, a table [10, 64] bf16 (1280 bytes), out [4, 2, 64] bf16 (1024 bytes)."""
    ok = dict(x=ctypes.c_void_p(0x1000000), dtype=0, T=4, H=2, d=64, xr=128, xh=64, pos=ctypes.c_void_p(0x2000000),
              cs=ctypes.c_void_p(0x3000000), tdtype=0, maxp=10, R=64, layout=0, inverse=0, out=FAR, orr=128, oh=64,
              stream=None)
    call = caller(lib.nrc_rope_rotate, ok)
    for out in (at(ok["pos"], 0), at(ok["pos"], 24), at(ok["pos"], -1022), at(ok["cs"], 0), at(ok["cs"], 1278),
                at(ok["cs"], -1022)):
        assert call(out=out) == EINVAL and b"apart" in lib.nrc_last_error(), hex(out.value)


# the operands of QUERIES, each in memory of its own, with their bytes: 6 rows of 8 heads, a cache of 8 blocks of 2 heads
# of 16 cells, 3 sequences of up to 4 blocks, a mask of a word a row
APART = dict(q=0x1000000, cache=0x2000000, tables=0x3000000, ctx=0x4000000, starts=0x5000000, mask=0x6000000)
SIZES = dict(q=6 * 512 * 2, cache=8 * 2 * 16 * 128 * 2, tables=3 * 4 * 4, ctx=12, starts=16, mask=6 * 8)


def places(start, size, own, unit):
    """Where `own` bytes, in steps of `unit`, meet [start, start + size): at its first byte, its last, from before it."""
    return start, start + (size - 1) // unit * unit, start - own + unit


def test_tree_attention_outputs_apart_from_the_inputs(lib):
    kw = {k: ctypes.c_void_p(v) for k, v in APART.items()}
    call = caller(lib.nrc_context_tree_attention, dict(QUERIES, out=FAR, lse=ctypes.c_void_p(0x20000000), ws=None,
                                                       ws_bytes=0, stream=None))
    for name in APART:
        for out in places(APART[name], SIZES[name], 6 * 8 * 128, 16):
            assert call(**kw, words=1, out=ctypes.c_void_p(out)) == EINVAL and b"apart" in lib.nrc_last_error(), (name, hex(out))
        for lse in places(APART[name], SIZES[name], 6 * 8 * 4, 4):
            assert call(**kw, words=1, lse=ctypes.c_void_p(lse)) == EINVAL and b"apart" in lib.nrc_last_error(), (name, hex(lse))
    # a split context's workspace
    long = dict(kw, max_ctx=100000, words=1)
    need = lib.nrc_context_tree_attention_workspace_bytes(3, 6, 8, 2, 2, 100000)
    assert need > 0
    inside = [p for name in APART for p in places(APART[name], SIZES[name], need, 16)]
    for ws in inside + [FAR.value, FAR.value + 6 * 8 * 128 - 16, FAR.value - need + 16, 0x20000000]:
        if ws > 0:
            assert call(**long, ws=ctypes.c_void_p(ws), ws_bytes=need) == EINVAL and b"apart" in lib.nrc_last_error(), hex(ws)


def test_attention_mass_out_apart_from_the_inputs(lib):
    """out [3, 2, 64] of strides 200 and 100: 564 floats from the first to the last."""
    kw = {k: ctypes.c_void_p(v) for k, v in APART.items()}
    lse = 0x7000000
    call = caller(lib.nrc_context_attention_mass, dict(QUERIES, lse=ctypes.c_void_p(lse), w=None, wb=0, wh=0, decay=1.0,
                                                       out=FAR, ob=200, oh=100, width=64, stream=None))
    for name, start in {**APART, "lse": lse}.items():
        for out in places(start, {**SIZES, "lse": 6 * 8 * 4}[name], 564 * 4, 4):
            assert call(**kw, words=1, out=ctypes.c_void_p(out)) == EINVAL and b"apart" in lib.nrc_last_error(), (name, hex(out))


def test_kv_evict_outputs_apart_from_each_other_and_the_inputs(lib):
    """3 sequences of 2 heads: 240 kept cells each of new_weights and new_positions, 3 new_lens, and a workspace."""
    from test_cache_ops_abi import PAGED

    names = ["cache", "tables", "lens", "w", "p", "ends", "nw", "np", "nl", "ws"]
    at = {n: 0x10000000 * (i + 1) for i, n in enumerate(names)}
    width, budget = 2400, 1200
    need = lib.nrc_context_kv_evict_workspace_bytes(3, 2, width, budget)
    assert need > 0
    size = dict(SIZES, lens=12, ends=12, w=4 * 6 * width, p=4 * 6 * width, nw=4 * 6 * budget, np=4 * 6 * budget, nl=12, ws=need)
    ok = dict(PAGED, lens=None, w=None, wb=2 * width, wh=width, p=None, pb=2 * width, ph=width, width=width, ends=None, sinks=0,
              recent=0, budget=budget, nw=None, np=None, nl=None, ws=None, ws_bytes=need, stream=None)
    ok.update({n: ctypes.c_void_p(a) for n, a in at.items()})
    call = caller(lib.nrc_context_kv_evict, ok)
    for out in ("nw", "np", "nl", "ws", "cache"):
        for other in names:
            if other == out:
                continue
            for place in places(at[other], size[other], size[out], 16 if out in ("ws", "cache") else 4):
                got = call(**{out: ctypes.c_void_p(place)})
                assert got == EINVAL and b"apart" in lib.nrc_last_error(), (out, other, hex(place))


def test_kv_evict_cells_in_memory_of_their_own(lib):
    """Strides (block, page, head) of 8 blocks of 2 heads of 16 cells of 128."""
    from test_cache_ops_abi import PAGED

    at = [ctypes.c_void_p(0x10000000 * i) for i in range(1, 9)]
    ok = dict(PAGED, cache=at[0], tables=at[1], lens=at[2], w=at[3], wb=128, wh=64, p=at[4], pb=128, ph=64, width=64,
              ends=at[5], sinks=0, recent=0, budget=40, nw=at[6], np=at[7], nl=FAKE, ws=None, ws_bytes=0, stream=None)
    call = caller(lib.nrc_context_kv_evict, ok)
    for bst, pst, hst in ((4096, 128, 0), (4096, 0, 2048), (0, 128, 2048), (4096, 120, 2048), (4096, 128, 2040),
                          (4088, 128, 2048), (2048, 128, 2048), (128, 128, 2048)):
        assert call(bst=bst, pst=pst, hst=hst) == EINVAL and b"overlap" in lib.nrc_last_error(), (bst, pst, hst)
    # one of a kind has no stride; an empty call is none
    assert call(bst=4096, pst=128, hst=0, B=0) == 0
    assert call(nb=1, bs=1, H=1, bst=0, pst=0, hst=0, nw=None) == EINVAL and b"NULL" in lib.nrc_last_error()
    # pages, heads and blocks in any order: refused for what comes after
    for kw in (dict(bst=4096, pst=256, hst=128), dict(bst=256, pst=2048, hst=128), dict(bst=128, pst=1024, hst=16384)):
        assert call(**kw, nw=None) == EINVAL and b"NULL" in lib.nrc_last_error(), kw


def test_rope_table_of_finite_values(lib):
    """Scalings and magnitudes that would make a table of NaN and infinities."""
    call = caller(lib.nrc_rope_table, dict(start=0, count=8, R=64, width=64, base=1e4, scaling=0, factor=1.0, orig=4096.0,
                                           low=1.0, high=2.0, magnitude=1.0, out=None, dtype=0, stream=None))
    for kw in (dict(scaling=1, factor=1e-310), dict(scaling=1, factor=1e-303), dict(scaling=2, factor=1e-306),
               dict(scaling=2, factor=1e-306, R=4, width=4), dict(scaling=3, factor=1e-309), dict(scaling=4, factor=1e-309),
               dict(magnitude=1e39), dict(magnitude=-1e39)):
        assert call(**kw) == EINVAL and b"finite" in lib.nrc_last_error(), kw
    for kw in (dict(scaling=1, factor=1e-3), dict(scaling=1, factor=1e300), dict(scaling=4, factor=64.0), dict(magnitude=3e38)):
        assert call(**kw) == EINVAL and b"NULL" in lib.nrc_last_error(), kw  # (refused for what comes after)
