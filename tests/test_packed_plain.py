"""The plain 64-bit forms that the GPU tests of packed sequences, the paged cache and rotary positions compare with
(tests/packed_util.py), pinned on the CPU to torch's softmax and autograd, to complex numbers and to worked numbers; and
what of rotary positions is made on the host."""
import copy
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import attend, check_gradients, check_one, gradients, places, turned  # noqa: E402


@pytest.fixture(scope="module")
def sa2():
    from block_sparse_attention_sa2_gb300 import build_lib
    if not build_lib.up_to_date():
        build_lib.build()
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    return m


def case(H=6, Hkv=2, n=9, m=21, d=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).bfloat16() for s in ((H, n, d), (Hkv, m, d), (Hkv, m, d), (H, n, d))]


@pytest.mark.parametrize("causal", [True, False])
def test_attention_is_softmax_attention(causal):
    q, k, v, _ = case()
    o, lse, a, ds = attend(q, k, v, causal, 0.2)
    kk, vv = (x.double().repeat_interleave(3, 0) for x in (k, v))
    s = torch.einsum("hnd,hmd->hnm", q.double(), kk) * 0.2
    if causal:
        for i in range(9):
            s[:, i, 21 - 9 + i + 1:] = -math.inf
    assert torch.allclose(o, torch.softmax(s, 2) @ vv, atol=1e-12)
    assert torch.allclose(lse, torch.logsumexp(s, 2), atol=1e-12)
    assert bool((a >= o.abs() - 1e-12).all()) and float(ds.max()) < 1e-3


@pytest.mark.parametrize("causal", [True, False])
def test_gradients_are_autograd(causal):
    q, k, v, do = case(n=15, m=15)
    x = [t.double().requires_grad_() for t in (q, k, v)]
    s = torch.einsum("hnd,hmd->hnm", x[0], x[1].repeat_interleave(3, 0)) / 8.0
    if causal:
        s = s + torch.full((15, 15), -math.inf, dtype=torch.float64).triu(1)
    want = torch.autograd.grad(((torch.softmax(s, 2) @ x[2].repeat_interleave(3, 0)) * do.double()).sum(), x)
    got, mags = gradients(q, k, v, do, causal)
    for g, w, a in zip(got, want, mags):
        assert torch.allclose(g, w, atol=1e-11) and bool((a >= g.abs() - 1e-11).all())


def test_the_checks_reject_a_wrong_result():
    q, k, v, do = case(n=40, m=64)
    o, lse, _, _ = attend(q, k, v)
    check_one(o.bfloat16(), lse.float(), q, k, v)
    for bad_o, bad_lse in ((o * torch.where(torch.arange(40) == 7, 1.05, 1.0)[:, None], lse), (o, lse + 1e-3),
                           (attend(q, k, v, False)[0], lse), (torch.where(o == o[0, 0, 0], math.nan, o), lse)):
        with pytest.raises(AssertionError):
            check_one(bad_o.bfloat16(), bad_lse.float(), q, k, v)
    q, k, v, do = case(n=64, m=64)
    want, _ = gradients(q, k, v, do)
    check_gradients([x.bfloat16() for x in want], q, k, v, do, [0, 64])
    for i in range(3):
        got = [x.bfloat16() for x in want]
        got[i] = got[i] * 1.05
        with pytest.raises(AssertionError):
            check_gradients(got, q, k, v, do, [0, 64])
    assert places([3, 0, 2], 1) == [1, 4, 4, 6]


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_turned_is_multiplication_by_complex_numbers(layout):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((2, 3, 5, 10), generator=g, dtype=torch.float64)
    pos = torch.randint(-9, 99, (2, 2, 5), generator=g)
    f, axis = [1.0, 0.1, 0.3, 2.0], [0, 0, 1, 1]
    y = turned(x, pos, f, axis, layout, 1.5)
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if layout == "interleaved" else (x[..., :4], x[..., 4:8])
    t = torch.stack([pos[i].double() * w for w, i in zip(f, axis)], -1)[:, None]
    z = torch.complex(a.contiguous(), b.contiguous()) * torch.polar(torch.full_like(t, 1.5), t)
    c, d = (y[..., 0:8:2], y[..., 1:8:2]) if layout == "interleaved" else (y[..., :4], y[..., 4:8])
    assert torch.allclose(c, z.real) and torch.allclose(d, z.imag) and torch.equal(y[..., 8:], x[..., 8:])
    back = turned(y, pos, f, axis, layout, 1 / 1.5, True)
    assert torch.allclose(back, x)


def test_frequencies(sa2):
    f = sa2.rotary_frequencies
    assert f(4) == [1.0, 10000.0**-0.5] and f(2, base=7.0) == [1.0]
    assert f(64, scaling="linear", factor=4.0) == [w / 4 for w in f(64)]
    b = f(64, scaling="base", factor=8.0)
    assert b[0] == 1.0 and math.isclose(b[-1], f(64)[-1] / 8, rel_tol=1e-12) and b == sorted(b, reverse=True)
    r = f(64, scaling="ramp", factor=8.0, trained=2048, fast=32, slow=1)
    for w, x in zip(f(64), r):
        turns = 2048 * w / (2 * math.pi)
        keep = 1.0 if turns >= 32 else 0.0 if turns <= 1 else (turns - 1) / 31
        assert math.isclose(x, w * keep + w / 8 * (1 - keep), rel_tol=1e-14)
    assert r[0] == 1.0 and math.isclose(r[-1], f(64)[-1] / 8)
    for bad in (dict(n=3), dict(n=0), dict(n=8, scaling="cubic"), dict(n=8, scaling="ramp", fast=1.0, slow=1.0)):
        with pytest.raises(ValueError):
            f(**bad)


def test_turns_are_exact(sa2):
    """frequency / (2 pi) modulo 1, to 2^-64 and the two roundings of 64-bit numbers that go before."""
    turns = sa2.load_library().sa2_rotary_turns
    # 2 pi to 40 digits
    tau = Fraction("6.283185307179586476925286766559005768394")
    for w in (0.0, 1.0, -1.0, 1e-4, 0.5, 3.0, 1e-300, 6.28, -7.5, 100.25, 2.0**-60):
        got = Fraction(turns(w) % 2**64, 2**64)
        want = Fraction(w) / tau
        off = (got - want) % 1
        off = min(off, 1 - off)
        assert off <= abs(want) * Fraction(3, 2**53) + Fraction(1, 2**53) * (1 if w < 0 or abs(w) > 6 else 0) + Fraction(1, 2**64), w
    assert turns(float("nan")) == 0 and turns(float("inf")) == 0


def test_rotary_refusals_and_copies(sa2):
    f = sa2.rotary_frequencies(64)
    r = sa2.Rotary(128, f, axes=[20, 12], layout="half", gain=1.25, device="cpu")
    assert r._pairs.tolist()[20][1] == 1 and r._pairs.tolist()[19][1] == 0 and r._pairs.shape == (32, 2)
    c = copy.deepcopy(r)
    assert c.axes == (20, 12) and c.gain == 1.25 and torch.equal(c._pairs, r._pairs) and c._pairs is not r._pairs
    for bad in (dict(d=100), dict(d=0), dict(d=2048), dict(d=56), dict(frequencies=[]), dict(frequencies=[math.nan] * 8),
                dict(frequencies=[1.0] * 12, layout="half"), dict(axes=[16, 15]), dict(axes=[32, 0]), dict(axes=[]), dict(layout="both"),
                dict(gain=math.inf)):
        with pytest.raises(ValueError):
            sa2.Rotary(**{**dict(d=128, frequencies=f, device="cpu"), **bad})
