"""Copies of a KvCache8 on the GPU: a deep copy grows by itself, a shallow one is the same cache."""
import copy

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cache8 import queries, random_cache, sa2  # noqa: E402,F401

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


def test_a_deep_copy_grows_by_itself(sa2):  # noqa: F811
    c = random_cache(sa2, 1, 2, 300, 64)
    d = copy.deepcopy(c)
    q, n = queries(1, 2, 3, 64, torch.bfloat16), torch.full((1,), 300, **I32)
    want = sa2.cache8_attn(q, c, n)
    held = [x.clone() for x in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    x = torch.ones((1, 2, 100, 64), dtype=torch.bfloat16, device="cuda")
    sa2.cache8_append(d, x, x, n - 100)
    sa2.check_device()
    assert all(torch.equal(a, b) for a, b in zip(held, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)))
    assert all(torch.equal(a, b) for a, b in zip(sa2.cache8_attn(q, c, n), want))
    k, v = sa2.cache8_read(d, n - 100, 100)
    assert torch.equal(k, x) and torch.equal(v, x)
    s = copy.copy(c)
    sa2.cache8_append(s, x, x, n - 100)
    k, _ = sa2.cache8_read(c, n - 100, 100)
    sa2.check_device()
    assert torch.equal(k, x)
