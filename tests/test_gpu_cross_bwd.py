"""Cross attention's gradient (sa2_cross_attn_bwd) against the formulas in 64 bits and against
differences of the 64-bit forward (tests/cross_util.py, which derives the bounds)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import attention, check_forward, check_gradients, gradients, lengths  # noqa: E402
from tests.test_gpu_cross import tensors  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    return m


def run(sa2, q, k, v, kv_len=None, scale=None, norm=True, check=True):
    """Forward and backward with NaN behind the lengths and in the gradients before the call."""
    B, M = q.shape[0], k.shape[2]
    lens = lengths(kv_len, B, M)
    kl = None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    k, v = k.clone(), v.clone()
    for b, n in enumerate(lens):
        k[b, :, n:] = math.nan
        v[b, :, n:] = math.inf
    g = torch.Generator(device="cuda").manual_seed(99)
    do = torch.randn(q.shape, generator=g, device="cuda").to(q.dtype)
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl, scale=scale)
    grads = [torch.full_like(x, math.nan) for x in (q, k, v)]
    sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=kl, scale=scale, dq=grads[0], dk=grads[1], dv=grads[2])
    sa2.check_device()
    if check:
        check_gradients(grads, q, k, v, do, lens, scale, norm)
    return grads, do


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 400])
@pytest.mark.parametrize("M", [2, 16, 17, 64, 65, 128, 129, 300])
def test_sizes(sa2, N, M, d):
    run(sa2, *tensors(2, 2, 2, N, M, d, torch.bfloat16, seed=N * 1000 + M), norm=M >= 64 and N >= 127)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (7, 1), (16, 2), (64, 1), (5, 1), (24, 8)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_heads(sa2, H, Hkv, d):
    run(sa2, *tensors(2, H, Hkv, 201, 200, d, torch.bfloat16, seed=H), kv_len=[200, 131])


@pytest.mark.parametrize("kv_len", [[0, 1, 2, 77], [77, 0, 0, 0], [0, 0, 0, 0], [64, 65, 63, 16]])
def test_padded_batch(sa2, kv_len):
    run(sa2, *tensors(4, 4, 2, 150, 300, 64, torch.bfloat16, seed=3), kv_len=kv_len, norm=False)


@pytest.mark.parametrize("d", [64, 128])
def test_one_key_has_no_score_gradient(sa2, d):
    """softmax of one score is 1: dS = 0, so dQ = dK = 0 up to rounding, and dV = sum dO."""
    run(sa2, *tensors(1, 3, 3, 200, 1, d, torch.bfloat16, seed=1), norm=False)


def test_many_pieces(sa2):
    """Key blocks whose query tiles several CTAs share, others that one CTA has whole, and more
    query tiles than CTAs."""
    run(sa2, *tensors(2, 3, 3, 3000, 520, 128, torch.bfloat16, seed=9), kv_len=[520, 200])
    run(sa2, *tensors(4, 16, 16, 300, 700, 64, torch.bfloat16, seed=10), kv_len=[700, 0, 129, 1])
    run(sa2, *tensors(3, 30, 10, 900, 1500, 64, torch.bfloat16, seed=11), kv_len=[1500, 77, 1111])


def test_token_major_and_fused(sa2):
    run(sa2, *tensors(2, 8, 4, 333, 190, 128, torch.bfloat16, seed=4, token_major=True), kv_len=[190, 100])
    g = torch.Generator(device="cuda").manual_seed(5)
    B, H, N, M, d = 2, 4, 200, 90, 64
    kv = torch.randn((B, M, 2 * H * d + 8), generator=g, device="cuda").bfloat16()
    q = torch.randn((B, N, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2)
    k = kv[:, :, :H * d].view(B, M, H, d).transpose(1, 2)
    v = kv[:, :, H * d:2 * H * d].view(B, M, H, d).transpose(1, 2)
    do = torch.randn((B, H, N, d), generator=g, device="cuda").bfloat16()
    # gradients into one buffer with the projection's layout; the gap stays as it was
    gkv = torch.full_like(kv, 5.0)
    dk = gkv[:, :, :H * d].view(B, M, H, d).transpose(1, 2)
    dv = gkv[:, :, H * d:2 * H * d].view(B, M, H, d).transpose(1, 2)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    dq, _, _ = sa2.cross_attn_bwd(q, k, v, o, lse, do, dk=dk, dv=dv)
    sa2.check_device()
    check_gradients((dq, dk, dv), q, k, v, do, [M] * B)
    assert bool((gkv[:, :, 2 * H * d:] == 5).all())


def test_scale(sa2):
    q, k, v = tensors(1, 2, 2, 300, 260, 128, torch.bfloat16, seed=6)
    run(sa2, q, k, v, scale=0.3, norm=False)
    run(sa2, q, k, v, scale=1e-3)


def test_against_differences(sa2):
    """The directional derivative of sum(O * dO) by central differences of the 64-bit forward."""
    q, k, v = tensors(2, 4, 2, 130, 140, 64, torch.bfloat16, seed=12)
    lens = [140, 70]
    grads, do = run(sa2, q, k, v, kv_len=lens)
    _, mags = gradients(q, k, v, do, lens)
    g = torch.Generator(device="cuda").manual_seed(13)
    h, u = 1e-5, 2.0**-8
    for i in range(3):
        x = [q.double(), k.double(), v.double()]
        dirn = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        loss = []
        for sgn in (1, -1):
            y = list(x)
            y[i] = x[i] + sgn * h * dirn
            loss.append(float((attention(*y, lens)[0] * do.double()).sum()))
        want = (loss[0] - loss[1]) / (2 * h)
        got = float((grads[i].double() * dirn).sum())
        bound = float(((u * grads[i].double().abs() + 3 * u * mags[i]) * dirn.abs()).sum())
        assert abs(got - want) <= 0.05 * bound + 1e-4 * abs(want), (i, got, want, bound)


def test_repeated_calls_are_identical(sa2):
    q, k, v = tensors(2, 6, 3, 1000, 400, 128, torch.bfloat16, seed=7)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    do = torch.randn_like(q)
    first = sa2.cross_attn_bwd(q, k, v, o, lse, do)
    for _ in range(20):
        again = sa2.cross_attn_bwd(q, k, v, o, lse, do)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    sa2.check_device()


def test_step_in_a_graph(sa2):
    """Forward and backward captured together, replayed on new inputs and lengths."""
    q, k, v = tensors(2, 4, 2, 300, 260, 64, torch.bfloat16, seed=8)
    do = torch.randn_like(q)
    kl = torch.tensor([260, 100], dtype=torch.int32, device="cuda")
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=kl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
        grads = sa2.cross_attn_bwd(q, k, v, o, lse, do, kv_len=kl)
    new = tensors(2, 4, 2, 300, 260, 64, torch.bfloat16, seed=18)
    for dst, src in zip((q, k, v), new):
        dst.copy_(src)
    do.copy_(torch.randn_like(do))
    kl.copy_(torch.tensor([0, 259], dtype=torch.int32))
    g.replay()
    sa2.check_device()
    check_forward(o, lse, *new, [0, 259])
    check_gradients(grads, *new, do, [0, 259])


def test_refusals(sa2):
    q, k, v = tensors(1, 2, 2, 64, 100, 64, torch.float16)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    with pytest.raises(sa2.Sa2Error):  # fp16 has no backward
        sa2.cross_attn_bwd(q, k, v, o, lse, o)
    q, k, v = tensors(1, 2, 2, 64, 100, 64, torch.bfloat16)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    for kw in (dict(do=o[:, :, :5]), dict(do=o.float()), dict(dk=torch.empty_like(q)), dict(lse=lse[:, :1])):
        with pytest.raises(ValueError):
            sa2.cross_attn_bwd(**{**dict(q=q, k=k, v=v, o=o, lse=lse, do=o), **kw})
    with pytest.raises(sa2.Sa2Error):
        sa2.cross_attn_bwd(q, k, v, o, lse, o, ws=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert sa2.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_captured_and_repeated(sa2, d):
    """A training step captured and replayed on new inputs, and calls that follow each other on one
    workspace: the kernels of a call may start before the one before them has ended."""
    shapes = [(2, 6, 2, 130, 300), (1, 2, 2, 17, 70), (1, 12, 12, 700, 129)]
    for B, H, Hkv, N, M in shapes:
        q, k, v = tensors(B, H, Hkv, N, M, d, torch.bfloat16, seed=N)
        do = torch.randn_like(q)
        ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        held = [x.clone() for x in (q, k, v, do)]
        grads = [torch.empty_like(x) for x in held[:3]]

        def step():
            o, lse = sa2.cross_attn_fwd(*held[:3])
            sa2.cross_attn_bwd(*held[:3], o, lse, held[3], dq=grads[0], dk=grads[1], dv=grads[2], ws=ws)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for i in range(1, 9):
            for x, y in zip(held, (q, k, v, do)):
                x.copy_(y * (1 + i / 8))
            graph.replay()
            replayed = [x.clone() for x in grads]
            for x in grads:
                x.fill_(math.nan)
            for _ in range(3):
                step()
            assert all(torch.equal(x, y) for x, y in zip(replayed, grads)), (N, M, i)
    sa2.check_device()
