"""Token strides that lie far apart: only strides that are used, and as they are used, are limited."""
import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import check_forward, check_gradients  # noqa: E402
from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def far(x, stride_n, stride_h):
    """x's values with tokens stride_n and heads stride_h elements apart."""
    B, H, n, d = x.shape
    assert B == 1
    y = torch.empty((n - 1) * stride_n + (H - 1) * stride_h + d + 8, dtype=x.dtype, device=x.device)
    y = y.as_strided((1, H, n, d), (8, stride_h, stride_n, 1))
    y.copy_(x)
    return y


@pytest.mark.parametrize("H,Hkv,N", [(40, 1, 2), (3, 1, 2), (2, 2, 3)])
def test_one_sequence(sa2, H, Hkv, N):  # noqa: F811
    """tokens x stride_n beyond 2^33 elements with a batch of one: the batch stride is no one's."""
    q, k, v = tensors(1, H, Hkv, N, 2, 128, torch.bfloat16, seed=H)
    do = torch.randn_like(q)
    fq, fk = far(q, 2**32, 128), far(k, 2**32, 128)
    o, lse = sa2.cross_attn_fwd(fq, fk, v)
    sa2.check_device()
    check_forward(o, lse, q, k, v, [2])
    grads = sa2.cross_attn_bwd(fq, fk, v, o, lse, do)
    sa2.check_device()
    check_gradients(grads, q, k, v, do, [2], norm=False)


def test_heads_far_apart(sa2):  # noqa: F811
    """A head stride of 2^33 elements, of keys that no other head shares."""
    q, k, v = tensors(1, 2, 2, 40, 70, 64, torch.bfloat16, seed=3)
    fk = far(k, 64, 2**33)
    o, lse = sa2.cross_attn_fwd(q, fk, v)
    sa2.check_device()
    check_forward(o, lse, q, k, v, [70])
