"""Cross attention of more than 65535 key heads in all (batch x heads): each within the stated limits."""
import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import check_forward, check_gradients  # noqa: E402
from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,N,M", [(5, 5, 1, 3), (6, 3, 2, 130)])
def test_forward_and_backward(sa2, H, Hkv, N, M):  # noqa: F811
    B = 65536 // Hkv + 77
    q, k, v = tensors(B, H, Hkv, N, M, 64, torch.bfloat16, seed=1)
    do = torch.randn_like(q)
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, M + 1, (B,), generator=g)
    kl = lens.to(device="cuda", dtype=torch.int32)
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=kl, dq=grads[0], dk=grads[1], dv=grads[2])
    sa2.check_device()
    at = torch.cat((torch.arange(3), torch.randint(0, B, (30,), generator=g), torch.arange(B - 3, B)))
    some = [int(x) for x in lens[at]]
    check_forward(o[at], lse[at], q[at], k[at], v[at], some)
    assert all(bool(x.isfinite().all()) for x in grads)
    check_gradients([x[at] for x in grads], q[at], k[at], v[at], do[at], some, norm=False)
