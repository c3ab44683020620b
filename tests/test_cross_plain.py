"""The plain 64-bit forms that the GPU tests compare with (tests/cross_util.py), pinned on the CPU to
torch's own softmax, autograd and float8 conversion, and to hand-worked scales."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import (BLOCK, HostCache, attention, cache_values, check_forward, check_gradients,  # noqa: E402
                              exponent, gradients, round_e4m3)


def case(B=2, H=6, Hkv=2, N=9, M=21, d=64, dtype=torch.bfloat16, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g).to(dtype) for s in ((B, H, N, d), (B, Hkv, M, d), (B, Hkv, M, d), (B, H, N, d))]


def test_attention_is_softmax_attention():
    q, k, v, _ = case()
    lens = [21, 8]
    o, lse, a, ds = attention(q, k, v, lens, 0.2)
    for b, n in enumerate(lens):
        kk, vv = (x[b, :, :n].double().repeat_interleave(3, 0) for x in (k, v))
        s = torch.einsum("hnd,hmd->hnm", q[b].double(), kk) * 0.2
        assert torch.allclose(o[b], torch.softmax(s, 2) @ vv, atol=1e-12)
        assert torch.allclose(lse[b], torch.logsumexp(s, 2), atol=1e-12)
    assert bool((a >= o.abs() - 1e-12).all()) and float(ds.max()) < 1e-3


def test_rows_without_keys():
    q, k, v, do = case()
    o, lse, _, _ = attention(q, k, v, [0, 5])
    assert bool((o[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    (dq, dk, dv), _ = gradients(q, k, v, do, [0, 5])
    assert not dq[0].any() and not dk[0].any() and not dv[0].any() and not dk[1, :, 5:].any()


def test_gradients_are_autograd():
    q, k, v, do = case()
    lens = [21, 8]
    x = [t.double().requires_grad_() for t in (q, k, v)]
    total = 0.0
    for b, n in enumerate(lens):
        kk, vv = (t[b, :, :n].repeat_interleave(3, 0) for t in x[1:])
        p = torch.softmax(torch.einsum("hnd,hmd->hnm", x[0][b], kk) / 8.0, 2)
        total = total + ((p @ vv) * do[b].double()).sum()
    want = torch.autograd.grad(total, x)
    got, mags = gradients(q, k, v, do, lens)
    for g, w, a in zip(got, want, mags):
        assert torch.allclose(g, w, atol=1e-11)
        assert bool((a >= g.abs() - 1e-11).all())


def test_the_checks_reject_a_wrong_result():
    q, k, v, do = case(N=40, M=64)
    lens = [64, 64]
    o, lse, _, _ = attention(q, k, v, lens)
    check_forward(o.bfloat16(), lse.float(), q, k, v, lens)
    bad = o.clone()
    bad[1, 2, 3] *= 1.05
    with pytest.raises(AssertionError):
        check_forward(bad.bfloat16(), lse.float(), q, k, v, lens)
    with pytest.raises(AssertionError):  # one key too many
        check_forward(o.bfloat16(), lse.float(), q, k, v, [64, 63])
    g, _ = gradients(q, k, v, do, lens)
    check_gradients([x.bfloat16() for x in g], q, k, v, do, lens)
    with pytest.raises(AssertionError):  # D left out
        check_gradients([(g[0] * 1.02).bfloat16(), g[1].bfloat16(), g[2].bfloat16()], q, k, v, do, lens)


def test_round_e4m3_is_the_format():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    every = every[~every.isnan()].double()
    assert torch.equal(round_e4m3(every), every)
    x = torch.randn(20000, generator=torch.Generator().manual_seed(1)) * torch.logspace(-4, 2.6, 20000)
    x = x.clamp(-448, 448)
    assert torch.equal(round_e4m3(x.double()), x.to(torch.float8_e4m3fn).float().double())
    mid = (every[None] + every[:, None]).flatten() / 2  # ties among them
    mid = mid.float().double()
    assert torch.equal(round_e4m3(mid), mid.float().to(torch.float8_e4m3fn).float().double())


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.5, 1), (449.0, 1), (447.0, 0), (224.0, -1), (224.25, 0), (1.0, -8),
                                    (1.75, -8), (1.7500001, -7), (0.0, -100), (1e-38, -100), (3.3e38, 119),
                                    (2.0**127, 119), (2.0**100, 92)])
def test_exponents(amax, e):
    assert exponent(amax) == e


def test_host_cache_keeps_grown_blocks():
    c = HostCache(1, 1, 130, 64)
    x = torch.full((1, 1, 3, 64), 1.0)
    c.append(x, [62], [3])  # two tokens in block 0, which keeps 62 under 2^0 (1 needs 2^-8); one in block 1
    assert [int(e) for e in c.e[0, 0]] == [0, -8, 0]
    assert torch.equal(c.values()[0, 0, 62:65], x[0, 0].double())
    c.append(torch.full((1, 1, 2, 64), 1000.0), [64], [2])  # overwrites block 1 from its start: its own scale
    assert int(c.e[0, 0, 0]) == 0 and int(c.e[0, 0, 1]) == 2
    c.append(torch.full((1, 1, 1, 64), 0.01), [66], [1])  # smaller: the scale stays
    assert int(c.e[0, 0, 1]) == 2 and float(c.values()[0, 0, 66, 0]) == float(round_e4m3(torch.tensor(0.01 / 4).double())) * 4
    x8 = (c.x).to(torch.float32).to(torch.float8_e4m3fn)
    assert torch.equal(cache_values(x8, torch.exp2(c.e.float())), c.values())
    assert BLOCK == 64
