"""Attention over the cache where every score is next to nothing: the factor that takes a row's products to
its scores (softmax scale, the row's power of two, K's scale) lies below the smallest fp32 number, and the
keys behind the last one must still be left out.  Bounds as in tests/cross_util.py."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cache8 import attend, queries, random_cache, sa2  # noqa: E402,F401

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def zero_keys(m, B, H, C, d, first, seed):
    """A cache whose keys are zeros (scale 2^-100) from block `first` on; values of order 1."""
    c = random_cache(m, B, H, C, d, seed=seed, spread=1)
    z = torch.zeros((B, H, C - 64 * first, d), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(z.shape, generator=g, device="cuda").bfloat16()
    m.cache8_append(c, z, v, torch.full((B,), 64 * first, **I32))
    return c


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 30])
@pytest.mark.parametrize("first,n", [(0, 5), (0, 64), (1, 100), (2, 129), (3, 250)])
@pytest.mark.parametrize("exponent", [-33, -40, -100, -126])
def test_zero_keys_and_tiny_queries(sa2, exponent, first, n, N, d):  # noqa: F811
    q = queries(2, 4, N, d, torch.bfloat16, seed=n, amp=2.0**exponent)
    o, lse = attend(sa2, q, zero_keys(sa2, 2, 2, 256, d, first, n), [n, max(1, n - 3)])
    assert bool(o.isfinite().all()) and bool(lse.isfinite().all())


@pytest.mark.parametrize("N", [1, 30])
def test_long_caches_split_over_the_sms(sa2, N):  # noqa: F811
    q = queries(1, 4, N, 128, torch.bfloat16, seed=N, amp=2.0**-50)
    attend(sa2, q, zero_keys(sa2, 1, 2, 6000, 128, 20, N), [5999])


@pytest.mark.parametrize("N", [1, 30])
def test_tiny_softmax_scale(sa2, N):  # noqa: F811
    q = queries(1, 2, N, 64, torch.float16, seed=N)
    attend(sa2, q, zero_keys(sa2, 1, 2, 256, 64, 1, N), [100], scale=1e-30)
