"""Keys that are left out by an infinite channel (queries hold 1 there, keys 0 or -inf): whole blocks, warps'
steps and parts without a score above -inf, and rows with none at all, which get O = 0 and LSE = -inf as
sequences without keys do.  The 64-bit form takes the remaining keys alone."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import check_forward  # noqa: E402
from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 40, 300])
@pytest.mark.parametrize("M,kept", [(300, (280, 300)), (300, (70, 90)), (129, (0, 1)), (5000, (4990, 5000)), (5000, (0, 3)),
                                    (5000, (2500, 2600)), (64, (63, 64)), (300, (128, 256))])
def test_blocks_without_scores(sa2, M, kept, N, d, dtype):  # noqa: F811
    q, k, v = tensors(2, 4, 2, N, M, d, dtype, seed=M + N)
    q[..., 5] = 1.0
    k[..., 5] = 0.0
    lo, hi = kept
    rest = k[:, :, lo:hi].contiguous(), v[:, :, lo:hi].contiguous()
    k[:, :, :lo, 5] = -math.inf
    k[:, :, hi:, 5] = -math.inf
    o, lse = sa2.cross_attn_fwd(q, k, v)
    sa2.check_device()
    check_forward(o, lse, q, *rest, [hi - lo] * 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,M", [(1, 100), (1, 5000), (40, 100), (40, 5000), (300, 257)])
def test_rows_without_scores(sa2, N, M, d):  # noqa: F811
    q, k, v = tensors(2, 4, 2, N, M, d, torch.bfloat16, seed=M + N)
    q[..., 5] = 1.0
    k[..., 5] = 0.0
    k[1, 1, :, 5] = -math.inf  # query heads 2 and 3 of the second sequence
    o, lse = sa2.cross_attn_fwd(q, k, v)
    sa2.check_device()
    assert not bool(o[1, 2:].any()) and bool((lse[1, 2:] == -math.inf).all())
    check_forward(o[:, :2], lse[:, :2], q[:, :2], k[:, :1], v[:, :1], [M] * 2)
    check_forward(o[:1], lse[:1], q[:1], k[:1], v[:1], [M])


def test_nan_and_plus_infinity_are_not_hidden(sa2):  # noqa: F811
    for N, M in ((1, 300), (1, 5000), (40, 300), (40, 5000)):
        for bad in (math.nan, math.inf):
            q, k, v = tensors(1, 2, 2, N, M, 64, torch.bfloat16, seed=N)
            q[..., 5] = 1.0
            k[0, 1, 77, 5] = bad
            o, lse = sa2.cross_attn_fwd(q, k, v)
            sa2.check_device()
            assert bool(o[0, 1].isnan().all()) and not bool(lse[0, 1].isfinite().any())
            assert bool(o[0, 0].isfinite().all()) and bool(lse[0, 0].isfinite().all())
