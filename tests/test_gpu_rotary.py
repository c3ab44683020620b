"""Rotary positions on the GPU against their formula in 64 bits.

Bound per element: the output's rounding, u |y|; and of gain (|a| + |b|), the pair's magnitudes, 2^-20 for sine and
cosine (2 ulp of values up to 1 is 2^-22, the angle's place in its turn is held to 2^-31 of a half turn and then
rounded to 24 bits, which moves both by pi 2^-25) and the products' roundings (3 of 2^-24), and |angle| 2^-50 for the
frequency, which is a rounded number in both forms (2^-53 relative, and as turns 2^-52)."""
import copy
import math

import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import I32, U, turned  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    return m


def rnd(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def axis_of(r):
    return [a for a, n in enumerate(r.axes) for _ in range(n)]


def check(y, x, pos, r, inverse=False):
    """x, y [B, H, N, d], pos [axes, B, N]."""
    n = len(r.frequencies)
    ref = turned(x, pos, r.frequencies, axis_of(r), r.layout, r.gain, inverse)
    mag = torch.zeros_like(ref)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if r.layout == "interleaved" else (slice(0, n), slice(n, 2 * n))
    both = (x[..., ia].double().abs() + x[..., ib].double().abs()) * abs(r.gain)
    angle = torch.stack([pos[a].double().abs() * abs(w) for w, a in zip(r.frequencies, axis_of(r))], -1)[:, None]
    mag[..., ia] = mag[..., ib] = both * (2.0**-20 + angle * 2.0**-50)
    bound = U[x.dtype] * ref.abs() * (1 + 2.0**-6) + mag + (2.0**-25 if x.dtype == torch.float16 else 1e-38)
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), f"{float((err / bound).nan_to_num(math.inf).max()):.3f} of the bound"
    assert torch.equal(y[..., 2 * n:], x[..., 2 * n:])


TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout,d,rot", [(x, d, rot) for x in ("interleaved", "half") for d, rot in
                                          ((64, 64), (128, 128), (128, 64), (128, 48), (64, 16), (96, 96), (256, 160))] +
                         [("interleaved", 8, 8)])
def test_parts_of_the_head(sa2, dtype, layout, d, rot):
    r = sa2.Rotary(d, sa2.rotary_frequencies(rot), layout=layout)
    q, k = rnd((2, 77, 5, d), dtype, 0).transpose(1, 2), rnd((2, 3, 77, d), dtype, 1)
    pos = torch.randint(0, 5000, (2, 77), generator=torch.Generator().manual_seed(2)).to(**I32)
    y, z = sa2.rotary(r, pos, q, k)
    yi, zi = sa2.rotary(r, pos, q, k, inverse=True)
    sa2.check_device()
    assert y.shape == q.shape and y.stride() == q.stride() and y.dtype == dtype
    for got, x, inverse in ((y, q, False), (z, k, False), (yi, q, True), (zi, k, True)):
        check(got, x, pos[None], r, inverse)


@pytest.mark.parametrize("pairs", [1, 3, 5, 22, 31])
def test_odd_counts_of_interleaved_pairs(sa2, pairs):
    r = sa2.Rotary(64, sa2.rotary_frequencies(2 * pairs))
    x = rnd((1, 2, 33, 64), torch.bfloat16, pairs)
    x[..., 2 * pairs:] = float("nan") if pairs % 2 else 3.0  # channels behind are not touched, whatever they are
    pos = torch.arange(33, **I32)
    y = sa2.rotary(r, pos, x)
    sa2.check_device()
    if pairs % 2:
        assert bool(y[..., 2 * pairs:].isnan().all())
        x, y = x.nan_to_num(0.0), y.nan_to_num(0.0)
    check(y, x, pos[None, None], r)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("axes", [(64,), (22, 21, 21), (24, 40), (1, 1, 1, 61)])
def test_axes(sa2, layout, axes):
    f = [w for n in axes for w in sa2.rotary_frequencies(2 * n)]
    r = sa2.Rotary(128, f, axes=axes, layout=layout)
    x = rnd((2, 3, 100, 128), torch.bfloat16, 0)
    shape = (2, 100) if len(axes) == 1 else (len(axes), 2, 100)
    pos = torch.randint(-50, 1000, shape, generator=torch.Generator().manual_seed(1)).to(**I32)
    y = sa2.rotary(r, pos, x)
    sa2.check_device()
    check(y, x, pos.reshape(len(axes), 2, 100), r)
    # the same positions in each sequence
    y = sa2.rotary(r, pos[..., 0, :].contiguous(), x)
    sa2.check_device()
    check(y, x, pos[..., :1, :].expand(shape).reshape(len(axes), 2, 100), r)


@pytest.mark.parametrize("at", [0, 10**6, 2**24 + 1, 2**31 - 40, -(2**31), -5])
def test_far_positions(sa2, at):
    r = sa2.Rotary(64, sa2.rotary_frequencies(64))
    x = rnd((1, 1, 40, 64), torch.float32, 0)
    pos = (torch.arange(40) + at).to(**I32)
    y = sa2.rotary(r, pos, x)
    sa2.check_device()
    check(y, x, pos[None, None], r)


@pytest.mark.parametrize("scaling", ["linear", "base", "ramp"])
def test_scaled(sa2, scaling):
    f = sa2.rotary_frequencies(64, scaling=scaling, factor=8.0, trained=2048)
    r = sa2.Rotary(128, f, layout="half", gain=1.2)
    x = rnd((1, 4, 60, 128), torch.bfloat16, 0)
    pos = torch.arange(100000, 100060, **I32)
    check(sa2.rotary(r, pos, x), x, pos[None, None], r)
    check(sa2.rotary(r, pos, x, inverse=True), x, pos[None, None], r, True)
    sa2.check_device()


def test_negative_and_zero_frequencies(sa2):
    r = sa2.Rotary(8, [0.0, -1.0, 3.0, 1e-30], gain=-0.5)
    x, pos = rnd((1, 1, 50, 8), torch.float32, 0), torch.arange(-25, 25, **I32)
    check(sa2.rotary(r, pos, x), x, pos[None, None], r)
    sa2.check_device()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_in_place_and_packed(sa2, dtype, layout):
    """[H, T, d] of packed sequences; in place the result is the same and channels behind are not written."""
    r = sa2.Rotary(128, sa2.rotary_frequencies(64), layout=layout)
    q, k = rnd((501, 7, 128), dtype, 0).transpose(0, 1), rnd((501, 2, 128), dtype, 1).transpose(0, 1)
    pos = torch.cat([torch.arange(200), torch.arange(301)]).to(**I32)
    y, z = sa2.rotary(r, pos, q, k)
    check(y[None], q[None], pos[None, None], r)
    q2, k2 = q.clone(), k.clone()
    y2, z2 = sa2.rotary(r, pos, q2, k2, q_out=q2, k_out=k2)
    sa2.check_device()
    assert y2 is q2 and z2 is k2 and torch.equal(y2, y) and torch.equal(z2, z)


@pytest.mark.parametrize("B,N,H", [(1, 1, 1), (1, 3, 40), (3, 1, 8), (1, 4000, 40), (2, 5003, 3)])
def test_sizes(sa2, B, N, H):
    """From one word to more heads and tokens than a pass of the grid."""
    for layout in ("interleaved", "half"):
        r = sa2.Rotary(64, sa2.rotary_frequencies(32), layout=layout)
        x = rnd((B, H, N, 64), torch.bfloat16, N)
        pos = torch.arange(N, **I32)
        y = sa2.rotary(r, pos, x)
        sa2.check_device()
        check(y, x, pos[None, None].expand(1, B, N), r)


def test_gradient_against_differences(sa2):
    """The inverse is the transposed map: <g, turn x> = <inverse g, x>, with the gain."""
    for layout in ("interleaved", "half"):
        r = sa2.Rotary(64, sa2.rotary_frequencies(48), layout=layout, gain=1.3)
        x, g = rnd((1, 2, 30, 64), torch.float32, 0), rnd((1, 2, 30, 64), torch.float32, 1)
        pos = torch.arange(7, 37, **I32)
        dx = sa2.rotary(r, pos, g, inverse=True)
        e = rnd((1, 2, 30, 64), torch.float32, 2)
        # the map is linear: a difference over any step is exact but for roundings of 2^-20 of each term
        step = (sa2.rotary(r, pos, x + e).double() - sa2.rotary(r, pos, x - e).double()) / 2
        a, b = (step * g.double()).sum(), (dx.double() * e.double()).sum()
        assert abs(float(a - b)) <= 2.0**-19 * 2 * float(((x.abs() + 2 * e.abs()).double() * g.double().abs()).sum()) * 1.3
        # and of a loss, through the formula
        xx = x.double().requires_grad_()
        (want,) = torch.autograd.grad((turned(xx, pos[None, None], r.frequencies, axis_of(r), layout, 1.3) * g.double()).sum(), xx)
        check(dx, g, pos[None, None], r, True)
        assert float((dx.double() - want).abs().max()) <= 2.0**-19 * 1.3 * 2 * float(g.abs().max())


def test_refusals(sa2):
    f = sa2.rotary_frequencies(64)
    r = sa2.Rotary(128, f)
    x, pos = rnd((2, 3, 10, 128), torch.bfloat16, 0), torch.arange(10, **I32)
    for bad in (dict(pos=pos.long()), dict(pos=pos[:9].contiguous()), dict(pos=torch.zeros((3, 10), **I32)),
                dict(pos=pos.cpu()), dict(q=x[..., :64]), dict(q=x.double()), dict(q=x.transpose(2, 3)), dict(q=x[0, 0]),
                dict(k=x.half()), dict(k=x[:1]), dict(k=x[:, :, :5]), dict(q_out=x[:1]), dict(q_out=torch.empty_like(x, dtype=torch.float16))):
        with pytest.raises((ValueError, sa2.Sa2Error)):
            sa2.rotary(**{**dict(rotary=r, pos=pos, q=x), **bad})
    with pytest.raises(sa2.Sa2Error, match="alignment"):
        y = torch.empty(2 * 3 * 10 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 3, 10, 128)
        sa2.rotary(r, pos, y)
    with pytest.raises(sa2.Sa2Error, match="invalid"):  # the same memory under other strides
        z = rnd((1, 10, 10, 128), torch.bfloat16, 0)
        sa2.rotary(r, pos, z, q_out=z.transpose(1, 2))
    # no tokens: nothing to do
    assert sa2.rotary(r, pos[:0], x[:, :, :0]).shape == (2, 3, 0, 128)
    sa2.check_device()
    assert copy.deepcopy(r).frequencies == r.frequencies


def test_no_heads_are_refused(sa2):
    r, pos = sa2.Rotary(128, sa2.rotary_frequencies(128)), torch.arange(10, **I32)
    x = rnd((2, 3, 10, 128), torch.bfloat16, 0)
    for heads in ((x[:, :0], x), (x, x[:, :0])):
        with pytest.raises(ValueError, match="head"):
            sa2.rotary(r, pos, *heads)
