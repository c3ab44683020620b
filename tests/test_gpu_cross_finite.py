"""Cross attention's gradients at the sizes, lengths and scales where the other tests leave the norm out:
every element written, finite and within its bound, with NaN behind the lengths and in the outputs before."""
import pytest

torch = pytest.importorskip("torch")

from tests.cross_finite import check_all_finite, check_finite_gradients  # noqa: E402
from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401
from tests.test_gpu_cross_bwd import run  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 400])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 64, 65, 128, 129, 300])
def test_sizes(sa2, N, M, d):  # noqa: F811
    check_all_finite(run(sa2, *tensors(2, 2, 2, N, M, d, torch.bfloat16, seed=N * 1000 + M), norm=False)[0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,N", [(4, 2, 150), (3, 1, 127), (7, 1, 40), (64, 1, 5)])
@pytest.mark.parametrize("kv_len", [[0, 1, 2, 77], [77, 0, 0, 0], [0, 0, 0, 0], [64, 65, 63, 16], [300, 129, 257, 1]])
def test_padded_batch(sa2, kv_len, H, Hkv, N, d):  # noqa: F811
    (dq, dk, dv), _ = run(sa2, *tensors(4, H, Hkv, N, 300, d, torch.bfloat16, seed=3), kv_len=kv_len, norm=False)
    check_all_finite((dq, dk, dv))
    for b, n in enumerate(kv_len):
        assert not bool(dk[b, :, n:].any()) and not bool(dv[b, :, n:].any()) and (n or not bool(dq[b].any()))


@pytest.mark.parametrize("scale", [0.3, 1e-3, 1e-12])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(sa2, scale, d):  # noqa: F811
    check_all_finite(run(sa2, *tensors(1, 2, 2, 300, 260, d, torch.bfloat16, seed=6), scale=scale, norm=False)[0])


def test_pieces(sa2):  # noqa: F811
    for B, H, Hkv, N, M, d, lens in ((2, 3, 3, 3000, 520, 128, [520, 200]), (4, 16, 16, 300, 700, 64, [700, 0, 129, 1]),
                                     (3, 30, 10, 900, 1500, 64, [1500, 77, 1111])):
        check_all_finite(run(sa2, *tensors(B, H, Hkv, N, M, d, torch.bfloat16, seed=9), kv_len=lens, norm=False)[0])


def test_after_the_sparse_attention(sa2):  # noqa: F811
    """The layer's step: gradients of cross attention on the sparse attention's output, token-major."""
    B, H, N, M, d = 2, 4, 1000, 77, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v, do = (torch.randn((B, N, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(4))
    tk, tv = (torch.randn((B, M, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(2))
    lens = [77, 20]
    kl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    bm = sa2.build_mask(q, k, 1.0, 1.0)
    o1, lse1 = sa2.attn_fwd(q, k, v, bm)
    o2, lse2 = sa2.cross_attn_fwd(o1, tk, tv, kv_len=kl)
    grads = [torch.full_like(x, float("nan")) for x in (o1, tk, tv)]
    sa2.cross_attn_bwd(o1, tk, tv, o2, lse2, do, kv_len=kl, dq=grads[0], dk=grads[1], dv=grads[2])
    got = sa2.attn_bwd(q, k, v, o1, lse1, grads[0], bm)
    sa2.check_device()
    check_finite_gradients(grads, o1, tk, tv, do, lens, norm=False)
    check_all_finite(got)
