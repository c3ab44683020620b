"""Lengths out of range in cross attention's backward: clamped, and reported, as the forward does."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu
BOUNDS = 7


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad,clamped", [([135, 60, 9], [130, 60, 9]), ([130, -1, 9], [130, 0, 9]), ([3, 4, 2**31 - 1], [3, 4, 130])])
def test_backward_reports_lengths(sa2, bad, clamped, d):  # noqa: F811
    q, k, v = tensors(3, 4, 2, 50, 130, d, torch.bfloat16, seed=2)
    do = torch.randn_like(q)
    good, kl = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (clamped, bad))
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=good)
    want = sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=good)
    assert sa2.device_status() == 0
    got = sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=kl)
    assert sa2.device_status() == BOUNDS
    assert all(torch.equal(a, b) for a, b in zip(got, want))
