"""Cross and cache attention as they are used together: a layer's step beside the sparse self attention,
encoder states kept in the cache over several steps, calls on several streams, failures, memory."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import attention, cache_values, check_forward, check_gradients  # noqa: E402
from tests.test_gpu_cross import tensors  # noqa: E402

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
TIMEOUT = 6


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    yield m
    m.debug_set_wait_limit(0, 0)


def test_layer_step(sa2):
    """Self attention under its block mask, then cross attention to text states of two lengths on its
    output, forward and backward: the chain's gradients are those of each part on the other's."""
    B, H, N, M, d = 2, 4, 1000, 77, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn((B, N, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(3))
    tk, tv = (torch.randn((B, M, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(2))
    do = torch.randn((B, N, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2)
    lens = [77, 20]
    kl = torch.tensor(lens, **I32)
    bm = sa2.build_mask(q, k, 1.0, 1.0)  # every block kept
    o1, lse1 = sa2.attn_fwd(q, k, v, bm)
    o2, lse2 = sa2.cross_attn_fwd(o1, tk, tv, kv_len=kl)
    d1, dtk, dtv = sa2.cross_attn_bwd(o1, tk, tv, o2, lse2, do, kv_len=kl)
    dq, dk, dv = sa2.attn_bwd(q, k, v, o1, lse1, d1, bm)
    sa2.check_device()
    check_forward(o2, lse2, o1, tk, tv, lens)
    check_gradients((d1, dtk, dtv), o1, tk, tv, do, lens, norm=False)
    # with every block kept the self attention is the dense one, which the cross attention also computes
    o3, lse3 = sa2.cross_attn_fwd(q, k, v)
    check_forward(o3, lse3, q, k, v, [N] * B)
    g3 = sa2.cross_attn_bwd(q, k, v, o3, lse3, d1)
    sa2.check_device()
    check_gradients(g3, q, k, v, d1, [N] * B)
    for a, b in zip((dq, dk, dv), g3):  # each within its roundings of the same gradient
        assert float((a.float() - b.float()).norm() / b.float().norm()) <= 4 * 2.0**-8


def test_encoder_states_kept_in_the_cache(sa2):
    """The states' keys and values go into the cache once and serve every step, beside another batch
    element whose states grow."""
    B, H, d = 2, 6, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    c = sa2.KvCache8.empty(B, 2, 640, d, "cuda")
    k, v = (torch.randn((B, 2, 512, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    pos, n_new = torch.zeros(B, **I32), torch.tensor([512, 257], **I32)
    sa2.cache8_append(c, k, v, pos, n_new)
    kl = n_new.clone()
    held = None
    for step in range(4):
        q = torch.randn((B, 200 if step % 2 else 2, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2)
        o, lse = sa2.cache8_attn(q, c, kl)
        sa2.check_device()
        rk, rv = sa2.cache8_read(c, torch.zeros(B, **I32), 257)
        if step:
            assert torch.equal(rk[0], held[0][0]) and torch.equal(rv[0], held[1][0])
        held = (rk, rv)
        kk, vv = cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale)
        lens = [512, 257 + 5 * step]
        check_forward(o, lse, q, kk, vv, lens, p_type=torch.float16, v_max=448 * float(c.v_scale[:, :, :5].max()))
        sa2.cache8_append(c, k[:, :, :5], v[:, :, :5], kl, torch.tensor([0, 5], **I32))
        kl[1] += 5


@pytest.mark.parametrize("H,Hkv,N", [(16, 1, 1), (17, 1, 1), (8, 1, 2), (4, 4, 16), (4, 4, 17), (6, 2, 5), (6, 2, 6)])
@pytest.mark.parametrize("d", [64, 128])
def test_both_sides_of_the_few_row_kernel(sa2, H, Hkv, N, d):
    """16 query rows per key head take one kernel, 17 the other: 16-bit keys and cached ones."""
    q, k, v = tensors(2, H, Hkv, N, 1300, d, torch.bfloat16, seed=H + N)
    kl = torch.tensor([1300, 61], **I32)
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    sa2.check_device()
    check_forward(o, lse, q, k, v, [1300, 61])
    c = sa2.KvCache8.empty(2, Hkv, 1300, d, "cuda")
    sa2.cache8_append(c, k, v, torch.zeros(2, **I32))
    o, lse = sa2.cache8_attn(q, c, kl)
    sa2.check_device()
    check_forward(o, lse, q, cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale), [1300, 61],
                  p_type=torch.float16, v_max=448 * float(c.v_scale.max()))


def test_scores_that_jump(sa2):
    """Keys whose scores exceed everything before them by more than P's type holds: the block's own
    maximum has to come first (2^100 and more in bf16, 2^14 in fp16)."""
    for dtype, jump in ((torch.bfloat16, 500.0), (torch.float16, 60.0)):
        q = torch.ones((1, 2, 40, 64), device="cuda", dtype=dtype)
        k = torch.zeros((1, 2, 600, 64), device="cuda", dtype=dtype)
        g = torch.Generator(device="cuda").manual_seed(3)
        v = torch.randn((1, 2, 600, 64), generator=g, device="cuda").to(dtype)
        for at, f in ((70, 0.25), (200, 0.5), (330, 1.0), (599, 0.9)):
            k[:, :, at] = f * jump / 64
        for n in (40, 2):
            o, lse = sa2.cross_attn_fwd(q[:, :, :n], k, v, scale=1.0)
            sa2.check_device()
            check_forward(o, lse, q[:, :, :n], k, v, [600], scale=1.0)
            c = sa2.KvCache8.empty(1, 2, 600, 64, "cuda")
            sa2.cache8_append(c, k, v, torch.zeros(1, **I32))
            o, lse = sa2.cache8_attn(q[:, :, :n], c, torch.tensor([600], **I32), scale=1.0)
            sa2.check_device()
            check_forward(o, lse, q[:, :, :n], cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale), [600],
                          scale=1.0, p_type=torch.float16, v_max=448 * float(c.v_scale.max()))


def test_value_scales_far_apart(sa2):
    """Blocks of values 2^80 apart: V's scale is in the exponent, so neither end leaves its range."""
    for N in (1, 30):
        c = sa2.KvCache8.empty(1, 1, 256, 64, "cuda")
        g = torch.Generator(device="cuda").manual_seed(4)
        x = torch.randn((1, 1, 256, 64), generator=g, device="cuda")
        for i, f in enumerate((2.0**-40, 2.0**40, 0.0, 1.0)):
            x[:, :, 64 * i:64 * i + 64] *= f
        k = torch.randn((1, 1, 256, 64), generator=g, device="cuda").bfloat16()
        sa2.cache8_append(c, k, x.bfloat16(), torch.zeros(1, **I32))
        q = torch.randn((1, 1, N, 64), generator=g, device="cuda").bfloat16()
        for n in (64, 128, 256):
            o, lse = sa2.cache8_attn(q, c, torch.tensor([n], **I32))
            sa2.check_device()
            kk, vv = cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale)
            check_forward(o, lse, q, kk, vv, [n], p_type=torch.float16, v_max=448 * float(c.v_scale[:, :, :n // 64].max()))


def test_value_scales_at_their_limits(sa2):
    """Values near the largest bf16 after a sequence of small ones whose scores are lower and lower."""
    for N in (1, 30):
        c = sa2.KvCache8.empty(1, 1, 512, 64, "cuda")
        g = torch.Generator(device="cuda").manual_seed(14)
        x = torch.randn((1, 1, 512, 64), generator=g, device="cuda").clamp(-3, 3)
        k = torch.zeros((1, 1, 512, 64), device="cuda")
        for i in range(8):  # scores rise by 30 from block to block, values by 2^15
            x[:, :, 64 * i:64 * i + 64] *= 2.0**(15 * i + 20)
            k[:, :, 64 * i:64 * i + 64] = i * 30.0 / 8
        sa2.cache8_append(c, k.bfloat16(), x.bfloat16(), torch.zeros(1, **I32))
        q = torch.ones((1, 1, N, 64), device="cuda", dtype=torch.bfloat16)
        for n, sgn in ((64, 1), (200, 1), (512, 1), (512, -1)):
            o, lse = sa2.cache8_attn(q * sgn, c, torch.tensor([n], **I32))
            sa2.check_device()
            kk, vv = cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale)
            s = torch.softmax((q[0, 0].double() * sgn) @ kk[0, 0, :n].T / 8, 1)
            # the reference is the largest of score + log2(scale): the tiny P of smaller ones are off by
            # 2^-25 of its scale times its weight
            top = (s.reshape(N, -1, n)[:, 0] * c.v_scale[0, 0].double().repeat_interleave(64)[:n]).amax() * 448
            check_forward(o, lse, q * sgn, kk, vv, [n], p_type=torch.float16, v_max=float(top))


def test_nan_and_infinity_in_use_stay_in_their_rows(sa2):
    """A NaN query row and an infinite one: only those rows' results are not finite."""
    q, k, v = tensors(1, 2, 2, 150, 300, 128, torch.bfloat16, seed=5)
    q[0, 1, 40, 3] = math.nan
    q[0, 0, 149, 3] = math.inf
    o, lse = sa2.cross_attn_fwd(q, k, v)
    sa2.check_device()
    bad = torch.zeros((1, 2, 150), dtype=torch.bool, device="cuda")
    bad[0, 1, 40] = bad[0, 0, 149] = True
    assert bool(o[bad].isnan().any(1).all()) and bool(o[~bad].isfinite().all()) and bool(lse[~bad].isfinite().all())
    clean = torch.where(bad[..., None], 0.0, q).to(q.dtype)
    o2, lse2 = sa2.cross_attn_fwd(clean, k, v)
    assert torch.equal(o2[~bad], o[~bad]) and torch.equal(lse2[~bad], lse[~bad])


def test_calls_at_the_same_time(sa2):
    """Split calls on two streams with workspaces of their own, and a graph beside eager calls."""
    a, b = (tensors(1, 4, 2, 40, 3000, 128, torch.bfloat16, seed=s) for s in (6, 7))
    want = [sa2.cross_attn_fwd(*x) for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = sa2.cross_attn_fwd(*a)
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for s, x in zip(streams, (a, b)):
            s.wait_stream(torch.cuda.current_stream())
            got.append(sa2.cross_attn_fwd(*x, stream=s))
        graph.replay()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for (o, lse), (wo, wl) in zip(got + [captured], want + [want[0]]):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    sa2.check_device()


def test_calls_keep_no_memory(sa2):
    q, k, v = tensors(1, 4, 2, 40, 3000, 64, torch.bfloat16, seed=8)
    c = sa2.KvCache8.empty(1, 2, 3000, 64, "cuda")
    pos = torch.zeros(1, **I32)

    def calls():
        o, lse = sa2.cross_attn_fwd(q, k, v)
        sa2.cross_attn_bwd(q, k, v, o, lse, o)
        sa2.cache8_append(c, k, v, pos)
        sa2.cache8_read(c, pos, 100)
        sa2.cache8_attn(q, c, pos + 3000)

    calls()
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(50):
        calls()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held


@pytest.mark.parametrize("which", ["forward", "split", "cache", "backward"])
def test_expired_wait_reports_timeout_and_the_context_survives(sa2, which):
    q, k, v = tensors(2, 4, 4, 300, 2000 if which == "split" else 400, 128, torch.bfloat16, seed=9)
    c = sa2.KvCache8.empty(2, 4, k.shape[2], 128, "cuda")
    sa2.cache8_append(c, k, v, torch.zeros(2, **I32))
    kl = torch.full((2,), k.shape[2], **I32)
    lens = [k.shape[2]] * 2
    o, lse = sa2.cross_attn_fwd(q, k, v)
    sa2.check_device()
    call = {"cache": lambda: sa2.cache8_attn(q, c, kl), "backward": lambda: sa2.cross_attn_bwd(q, k, v, o, lse, o)}.get(
        which, lambda: sa2.cross_attn_fwd(q, k, v))
    sa2.debug_set_wait_limit(2_000_000, 200_000_000)
    try:
        call()
        status = sa2.device_status()
    finally:
        sa2.debug_set_wait_limit(0, 0)
    assert status == TIMEOUT
    got = call()
    sa2.check_device()
    if which == "backward":
        check_gradients(got, q, k, v, o, lens)
    elif which == "cache":
        check_forward(*got, q, cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale), lens, p_type=torch.float16,
                      v_max=448 * float(c.v_scale.max()))
    else:
        check_forward(*got, q, k, v, lens)


def test_offsets_past_32_bits(sa2):
    """A cache and queries whose elements lie more than 2^32 bytes from the first: the last sequence."""
    B, Hkv, C, d = 2, 8, 1_200_000, 128  # 2.46 GB of keys per sequence pair, strides past 2^31
    c = sa2.KvCache8.empty(B, Hkv, C, d, "cuda")
    assert c.k.numel() > 2**31
    # the last piece begins inside a block: the tokens that the block keeps have to be defined
    for x8, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x8.view(torch.uint8).zero_()
        sc.fill_(2.0**-100)
    g = torch.Generator(device="cuda").manual_seed(10)
    n = 300
    k, v = (torch.randn((B, Hkv, n, d), generator=g, device="cuda").bfloat16() for _ in range(2))
    for start in (0, C - n):
        sa2.cache8_append(c, k, v, torch.full((B,), start, **I32))
    rk, rv = sa2.cache8_read(c, torch.full((B,), C - n, **I32), n)
    sa2.check_device()
    fk, fv = sa2.cache8_read(c, torch.zeros(B, **I32), n)
    lastk = cache_values(c.k[:, :, -128:], c.k_scale[:, :, -2:])  # two whole blocks: C is a multiple of 64
    assert C % 64 == 0 and torch.equal(rk[:, :, -128:].double(), lastk)
    q = torch.randn((B, Hkv, 20, d), generator=g, device="cuda").bfloat16()
    o, lse = sa2.cache8_attn(q, c, torch.full((B,), n, **I32))
    sa2.check_device()
    check_forward(o, lse, q, fk, fv, [n] * B, p_type=torch.float16, v_max=448 * float(c.v_scale[:, :, :5].max()))
    # attention over everything: the middle is zeros (score 0, value 0) under a scale of 2^-100
    for N in (1, 20):
        o, lse = sa2.cache8_attn(q[:, :, :N], c, torch.full((B,), C, **I32))
        sa2.check_device()
        head, tail = (cache_values(x[0][:, :, s], x[1][:, :, t]) for x in ((c.k, c.k_scale),)
                      for s, t in ((slice(0, 320), slice(0, 5)), (slice(C - 320, C), slice(C // 64 - 5, None))))
        hv, tv = (cache_values(x[0][:, :, s], x[1][:, :, t]) for x in ((c.v, c.v_scale),)
                  for s, t in ((slice(0, 320), slice(0, 5)), (slice(C - 320, C), slice(C // 64 - 5, None))))
        s = torch.einsum("bhnd,bhmd->bhnm", q[:, :, :N].double(), torch.cat((head, tail), 2)) / math.sqrt(d)
        total = torch.exp(s).sum(3) + (C - 640)
        want = torch.einsum("bhnm,bhmd->bhnd", torch.exp(s), torch.cat((hv, tv), 2)) / total[..., None]
        assert torch.allclose(lse.double(), torch.log(total), atol=1e-4)
        # O is 640 values' weighted sum over 1.2 million weights: P is in fp16 below 2^-14 of the largest
        # weight, so each term is off by 2^-11 of itself or 2^-25 of the largest weight
        m = torch.exp(s).amax(3, keepdim=True).clamp(min=1.0)
        a = torch.einsum("bhnm,bhmd->bhnd", torch.exp(s) * 2.0**-10 + m * 2.0**-25 * 256, torch.cat((hv, tv), 2).abs())
        bound = a / total[..., None] + want.abs() * 2.0**-8 + 448 * 2.0**-100
        assert float(((o.double() - want).abs() / bound).max()) <= 1.0
