"""Cross attention of values far from 1 under scores that leap: P may lead a row's reference only so far
that P V stays within fp32.  Bounds as in tests/cross_util.py."""
import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import check_forward  # noqa: E402
from tests.test_gpu_cross import sa2  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [2, 40, 300])
@pytest.mark.parametrize("value,leaps", [(2.0**100, [35.0]), (2.0**100, [9.0]), (2.0**100, [12.0]), (2.0**100, [30.0, 65.0]),
                                         (1e15, [62.0]), (1e30, [25.0, 30.0])])
def test_leaps_beside_large_values(sa2, value, leaps, N, d):  # noqa: F811
    """The first half block's scores are 0; keys 70, 200 .. lead it by `leaps` (natural units)."""
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q = torch.ones((1, 2, N, d), device="cuda", dtype=torch.bfloat16)
    k = torch.zeros((1, 2, 300, d), device="cuda", dtype=torch.bfloat16)
    for i, leap in enumerate(leaps):
        k[:, :, 70 + 130 * i] = leap / d
    v = (torch.randn((1, 2, 300, d), generator=g, device="cuda") * value).bfloat16()
    o, lse = sa2.cross_attn_fwd(q, k, v, scale=1.0)
    sa2.check_device()
    assert bool(o.isfinite().all())
    check_forward(o, lse, q, k, v, [300], scale=1.0)


@pytest.mark.parametrize("N", [2, 40])
def test_many_leading_keys(sa2, N):  # noqa: F811
    """Every key of the second half lies 2^14 and more above the first ones; long keys, split over the SMs."""
    g = torch.Generator(device="cuda").manual_seed(N)
    q = torch.ones((1, 2, N, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.zeros((1, 2, 4000, 64), device="cuda", dtype=torch.bfloat16)
    k[:, :, 2001:] = 10.0 / 64
    k[:, :, 1:2000:7] = 7.0 / 64
    v = (torch.rand((1, 2, 4000, 64), generator=g, device="cuda") * 2.0**100).bfloat16()
    o, lse = sa2.cross_attn_fwd(q, k, v, scale=1.0)
    sa2.check_device()
    check_forward(o, lse, q, k, v, [4000], scale=1.0)
