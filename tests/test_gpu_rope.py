"""rope_table and rope_rotate against 64-bit references."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def nrc():
    import norm_rope_cache_amd as m

    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    m._load()
    return m


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def frequencies(R, base, scaling, factor, orig, low, high):
    f = []
    for j in range(R // 2):
        b = base * factor ** (R / (R - 2)) if scaling == "base" else base
        v = b ** (-2.0 * j / R)
        turns = orig * v / (2 * math.pi)
        if scaling == "linear":
            v /= factor
        elif scaling == "bands":
            m = min(1.0, max(0.0, (turns - low) / (high - low)))
            v *= m + (1 - m) / factor
        elif scaling == "ramp":
            index = lambda t: math.log(orig / (t * 2 * math.pi)) / math.log(base) * R / 2
            a, z = max(0.0, math.floor(index(high))), min(R / 2 - 1, math.ceil(index(low)))
            m = min(1.0, max(0.0, (j - a) / max(z - a, 1e-3)))
            v *= 1 - m + m / factor
        f.append(v)
    return torch.tensor(f, dtype=torch.float64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands", "ramp"])
@pytest.mark.parametrize("R,width,count,start", [(64, 64, 1000, 0), (2, 2, 5, 0), (6, 64, 33, 12345), (128, 130, 17, 99990),
                                                 (256, 256, 1, 2 ** 28 - 1)])
def test_table(nrc, dtype, scaling, R, width, count, start):
    if R == 2 and scaling == "base":
        with pytest.raises(nrc.NrcError):
            nrc.rope_table(count, R, scaling=scaling, factor=2.0)
        return
    got = nrc.rope_table(count, R, base=500000.0, scaling=scaling, factor=8.0, original_max=8192, low=1.0, high=32.0,
                         magnitude=1.1, width=width, start=start, dtype=dtype)
    f = frequencies(R, 500000.0, scaling, 8.0, 8192, 1.0, 32.0)
    a = torch.arange(start, start + count, dtype=torch.float64)[:, None] * f
    half = width // 2
    want = torch.zeros(count, width, dtype=torch.float64)
    want[:, R // 2:half] = 1.0
    want[:, :R // 2], want[:, half:half + R // 2] = 1.1 * torch.cos(a), 1.1 * torch.sin(a)
    # angles of up to start + count radians: a frequency is off by 4 roundings of
    # 2^-53 (pow, the scaling) and their product by one, on both sides; the run's 16 steps
    # add 2^-50; one rounding to the type, after one to FP32
    angle = (start + count) * 10 * 2.0 ** -53 + 2.0 ** -48
    tol = want.abs() * (half_step(dtype) + 2.0 ** -24) + 1.1 * angle
    assert bool(((got.double().cpu() - want).abs() <= tol).all())


def test_table_feeds_the_store(nrc):
    """The table in the store's form equals the store's own (bf16 of cos and sin), up to roundings of ties."""
    from norm_rope_cache_amd import synth

    t = nrc.rope_table(4096, 64, base=10000.0)
    want = torch.from_numpy(synth.rope_table(4096).view("int16").copy()).view(torch.bfloat16)
    assert t.shape == want.shape
    # one step of bf16 at most where a value lies at a border of rounding
    assert bool(((t.cpu().float() - want.float()).abs() <= want.float().abs() * 2.0 ** -7 + 1e-9).all())


def rotate(x, positions, table, layout, inverse):
    R = table.shape[1]
    out = x.clone()
    row = table[positions][:, None, :]
    c, s = row[..., :R // 2], row[..., R // 2:] * (-1 if inverse else 1)
    ia, ib = (slice(0, R, 2), slice(1, R, 2)) if layout == "interleaved" else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    size = torch.zeros_like(x)
    size[..., ia], size[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, size


TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("table", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("T,H,d,R", [(1, 1, 2, 2), (5, 3, 64, 64), (17, 24, 128, 64), (3, 5, 80, 20), (33, 1, 96, 48),
                                     (2, 7, 66, 34), (130, 64, 64, 16), (7, 2, 512, 256)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotate(nrc, dtype, table, layout, T, H, d, R, inverse):
    gen = torch.Generator().manual_seed(T + H + d)
    x = torch.randn(T, H, d, generator=gen).to(dtype)
    pos = torch.randint(0, 500, (T,), generator=gen)
    cs = nrc.rope_table(500, R, dtype=table)
    want, size = rotate(x.double(), pos, cs.double().cpu(), layout, inverse)
    got = nrc.rope_rotate(x.cuda(), pos.cuda(), cs, layout=layout, inverse=inverse)
    # a product and an FMA (2^-24 each of the terms' size), then half a step of the type
    # (a subnormal's: half of the type's least value)
    tol = want.abs() * half_step(dtype) + size * 2 * 2.0 ** -24 * (1 + half_step(dtype)) + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert bool(((got.double().cpu() - want).abs() <= tol).all())
    assert torch.equal(got[..., R:].cpu(), x[..., R:])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("dtype", TYPES)
def test_rotate_views_in_place_and_unaligned(nrc, layout, dtype):
    """Columns of a wider row, in place; an odd offset takes the element path: the same bits."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(9, 4, 64, generator=gen).to(dtype).cuda()
    pos = torch.randint(0, 100, (9,), generator=gen).cuda()
    cs = nrc.rope_table(100, 64, dtype=torch.float32)
    want = nrc.rope_rotate(x, pos, cs, layout=layout)
    wide = torch.zeros(9, 6, 64, dtype=dtype, device="cuda")
    view = wide[:, 1:5]
    view.copy_(x)
    assert nrc.rope_rotate(view, pos, cs, layout=layout, out=view) is view
    assert torch.equal(view, want) and bool((wide[:, 0] == 0).all()) and bool((wide[:, 5] == 0).all())
    odd = torch.zeros(9, 4, 71, dtype=dtype, device="cuda")[..., 3:67]
    odd.copy_(x)
    assert torch.equal(nrc.rope_rotate(odd, pos, cs, layout=layout), want)
    by_head = torch.zeros(4, 9, 64, dtype=dtype, device="cuda").permute(1, 0, 2)
    assert torch.equal(nrc.rope_rotate(x, pos, cs, layout=layout, out=by_head), want)


def test_inverse_is_the_gradient(nrc):
    """Against the transposed formula, against central differences, and back again."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(6, 2, 12, generator=gen, dtype=torch.float64)
    g = torch.randn(6, 2, 12, generator=gen, dtype=torch.float64)
    pos = torch.randint(0, 50, (6,), generator=gen)
    cs = nrc.rope_table(50, 8, dtype=torch.float32)
    table = cs.double().cpu()
    for layout in ("interleaved", "half"):
        back = nrc.rope_rotate(g.float().cuda(), pos.cuda(), cs, layout=layout, inverse=True).double().cpu()
        leaf = x.clone().requires_grad_()
        ia, ib = (slice(0, 8, 2), slice(1, 8, 2)) if layout == "interleaved" else (slice(0, 4), slice(4, 8))
        row = table[pos][:, None, :]
        c, s = row[..., :4], row[..., 4:]
        a, b = leaf[..., ia], leaf[..., ib]
        ((a * c - b * s) * g[..., ia] + (b * c + a * s) * g[..., ib]).sum().add((leaf[..., 8:] * g[..., 8:]).sum()).backward()
        # g itself rounded to FP32, two terms, two roundings
        tol = 4 * 2.0 ** -24 * (g.abs().amax() * 2)
        assert bool(((back - leaf.grad).abs() <= tol).all())
        # the map is linear: differences of the kernel's own outputs over a step of 1, FP32
        f = lambda t: (nrc.rope_rotate(t.float().cuda(), pos.cuda(), cs, layout=layout).double().cpu() * g).sum()
        for i in range(12):
            e = torch.zeros_like(x)
            e[2, 1, i] = 1.0
            diff = (f(e) - f(-e)) / 2
            assert abs(float(diff - back[2, 1, i])) <= 8 * 2.0 ** -24 * float(g.abs().amax())


def test_rows_without_a_table_row_stay(nrc):
    x = torch.randn(4, 2, 64, dtype=torch.float32, device="cuda")
    cs = nrc.rope_table(10, 64, dtype=torch.float32)
    pos = torch.tensor([-1, 3, 10, 2 ** 40], device="cuda")
    out = torch.full_like(x, 5.0)
    nrc.rope_rotate(x, pos, cs, out=out)
    assert bool((out[[0, 2, 3]] == 5).all()) and not bool((out[1] == 5).any())


def test_values_that_are_not_finite(nrc):
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 4], x[0, 0, 8] = math.nan, math.inf
    cs = nrc.rope_table(10, 64)
    y = nrc.rope_rotate(x, torch.tensor([3], device="cuda"), cs)[0, 0].float().cpu()
    bad = {i for i in range(64) if not math.isfinite(float(y[i]))}
    assert bad == {4, 5, 8, 9}
    raw = nrc.rope_rotate(x, torch.tensor([3], device="cuda"), cs).view(torch.int16)[0, 0]
    assert int(raw[4]) == 0x7FC0


def test_graph_and_stream(nrc):
    x = torch.randn(50, 8, 64, device="cuda").to(torch.bfloat16)
    pos = torch.arange(50, device="cuda")
    want_t = nrc.rope_table(64, 64, scaling="linear", factor=2.0)
    want = nrc.rope_rotate(x, pos, want_t)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t = nrc.rope_table(64, 64, scaling="linear", factor=2.0)
        y = nrc.rope_rotate(x, pos, t)
    for _ in range(3):
        y.zero_()
        t.zero_()
        g.replay()
        nrc.rope_rotate(x, pos, want_t)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(t, want_t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = nrc.rope_rotate(x, pos, want_t, stream=s)
    s.synchronize()
    assert torch.equal(z, want)


def test_refusals(nrc):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    cs = nrc.rope_table(10, 64)
    bad = [dict(x=x.double()), dict(x=x.cpu()), dict(x=x[0]), dict(x=x.transpose(1, 2)), dict(positions=pos.int()),
           dict(positions=pos[:3]), dict(positions=pos.cpu()), dict(positions=None), dict(cos_sin=None), dict(cos_sin=cs.half()), dict(cos_sin=cs.cpu()),
           dict(cos_sin=cs[:, ::2]), dict(cos_sin=nrc.rope_table(10, 128)), dict(layout="pairs"),
           dict(out=torch.zeros(4, 2, 64, device="cuda")), dict(out=x[:3])]
    for kw in bad:
        with pytest.raises((ValueError, TypeError, nrc.NrcError)):
            nrc.rope_rotate(**{**dict(x=x, positions=pos, cos_sin=cs), **kw})
    buf = torch.zeros(4, 2, 72, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(nrc.NrcError):  # overlaps x without being x
        nrc.rope_rotate(buf[..., :64], pos, cs, out=buf[..., 8:])
    with pytest.raises(nrc.NrcError):  # its own heads in one place
        nrc.rope_rotate(x, pos, cs, out=torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda").expand(4, 2, 64))
    for kw in (dict(count=-1), dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(width=62), dict(width=65),
               dict(base=1.0), dict(base=math.nan), dict(scaling="other"), dict(scaling="linear", factor=0.0),
               dict(scaling="ramp", factor=2.0, original_max=0), dict(scaling="bands", factor=2.0, original_max=9, low=2.0, high=1.0),
               dict(magnitude=math.inf), dict(start=-1), dict(start=2 ** 28), dict(start=2 ** 64), dict(dtype=torch.float16), dict(device="cpu"),
               dict(out=torch.zeros(4, 64, device="cuda"))):
        with pytest.raises((ValueError, TypeError, RuntimeError, nrc.NrcError)):
            nrc.rope_table(**{**dict(count=10, rotary_dim=64), **kw})
    assert nrc.rope_rotate(x[:0], pos[:0], cs).shape == (0, 2, 64)
    assert nrc.rope_table(0, 64).shape == (0, 64)
