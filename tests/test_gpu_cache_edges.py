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
