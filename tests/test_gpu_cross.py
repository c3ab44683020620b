"""Cross attention forward (sa2_cross_attn_fwd) against a plain 64-bit form (tests/cross_util.py, which
derives the bounds)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import check_forward, lengths  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    return m


def tensors(B, H, Hkv, N, M, d, dtype, seed=0, token_major=False, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(heads, n):
        if token_major:
            return (torch.randn((B, n, heads, d), generator=g, device="cuda") * amp).to(dtype).transpose(1, 2)
        return (torch.randn((B, heads, n, d), generator=g, device="cuda") * amp).to(dtype)

    return make(H, N), make(Hkv, M), make(Hkv, M)


def run(sa2, q, k, v, kv_len=None, scale=None):
    """One call with a workspace and outputs that start as NaN; checks every row."""
    B, M = q.shape[0], k.shape[2]
    lens = lengths(kv_len, B, M)
    kl = None if kv_len is None else torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    k, v = k.clone(), v.clone()
    for b, n in enumerate(lens):
        k[b, :, n:] = math.nan
        v[b, :, n:] = math.inf
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, dtype=torch.float32, device="cuda")
    sa2.cross_attn_fwd(q, k, v, kv_len=kl, scale=scale, o=o, lse=lse)
    sa2.check_device()
    check_forward(o, lse, q, k, v, lens, scale)
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 300])
@pytest.mark.parametrize("M", [1, 15, 16, 17, 64, 65, 127, 128, 129, 257])
def test_sizes(sa2, N, M, d):
    run(sa2, *tensors(2, 3, 3, N, M, d, torch.bfloat16, seed=N * 1000 + M))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (7, 1), (16, 2), (64, 1), (5, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_shared_key_heads(sa2, H, Hkv, d, dtype):
    run(sa2, *tensors(2, H, Hkv, 77, 200, d, dtype, seed=H), kv_len=[200, 131])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kv_len", [[0, 1, 2, 77], [77, 0, 0, 0], [0, 0, 0, 0], [64, 65, 63, 16]])
def test_padded_batch(sa2, kv_len, dtype):
    run(sa2, *tensors(4, 4, 4, 150, 77, 64, dtype, seed=3), kv_len=kv_len)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,M,kv_len", [(1, 3000, None), (64, 5000, [5000, 1]), (40, 4097, [0, 4097]),
                                        (129, 2000, [1999, 700]), (300, 1025, [1025, 1024]), (3, 1100, [0, 0])])
def test_keys_split_over_the_sms(sa2, N, M, kv_len, d):
    """Few queries over many keys: parts of a row's keys come from several CTAs."""
    B = 1 if kv_len is None else 2
    run(sa2, *tensors(B, 6, 2, N, M, d, torch.bfloat16, seed=M), kv_len=kv_len)


def test_many_segments_per_cta(sa2):
    """More query tiles than CTAs, key blocks from none to five: the rings run on across tiles."""
    run(sa2, *tensors(5, 16, 16, 2100, 520, 64, torch.bfloat16, seed=9), kv_len=[520, 0, 129, 1, 384])
    run(sa2, *tensors(3, 24, 8, 1000, 300, 128, torch.bfloat16, seed=10), kv_len=[300, 13, 256])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv_len", [None, [300, 0], [1, 129]])
def test_last_round_of_single_tiles(sa2, kv_len, d):
    """A few tile pairs more than SMs: those go tile by tile, the last pair of each head has one tile only."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    pairs = (sms + 12) // 4  # times 2 x 2 heads: 8 to 12 segments behind the first round
    run(sa2, *tensors(2, 2, 2, (2 * pairs - 1) * 128 - 5, 300, d, torch.bfloat16, seed=21), kv_len=kv_len)


def test_token_major_tensors(sa2):
    run(sa2, *tensors(2, 8, 4, 333, 190, 128, torch.bfloat16, seed=4, token_major=True), kv_len=[190, 100])


def test_strides_of_a_fused_projection(sa2):
    """q, k, v as slices of wider tensors: every tensor with strides of its own."""
    g = torch.Generator(device="cuda").manual_seed(5)
    B, H, N, M, d = 2, 4, 200, 90, 64
    wide = torch.randn((B, N, 3 * H * d), generator=g, device="cuda").bfloat16()
    kv = torch.randn((B, M, 2 * H * d + 8), generator=g, device="cuda").bfloat16()
    q = wide[:, :, H * d:2 * H * d].view(B, N, H, d).transpose(1, 2)
    k = kv[:, :, :H * d].view(B, M, H, d).transpose(1, 2)
    v = kv[:, :, H * d:2 * H * d].view(B, M, H, d).transpose(1, 2)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    sa2.check_device()
    assert o.shape == q.shape
    check_forward(o, lse, q, k, v, [M] * B)
    # an output with gaps between its rows: they stay as they were
    buf = torch.full((B, N, H, d + 64), 7.0, device="cuda", dtype=torch.bfloat16)
    sa2.cross_attn_fwd(q, k, v, o=buf[..., :d].transpose(1, 2))
    sa2.check_device()
    assert torch.equal(buf[..., :d].transpose(1, 2), o) and bool((buf[..., d:] == 7).all())


def test_scale_and_large_scores(sa2):
    q, k, v = tensors(1, 2, 2, 200, 600, 128, torch.bfloat16, seed=6, amp=4.0)
    run(sa2, q, k, v, scale=0.5)
    run(sa2, q, k, v, scale=1e-3)
    # a maximum that keeps growing along the keys: the running maximum is rescaled again and again
    ramp = torch.linspace(0, 8, 600, device="cuda")[None, None, :, None].bfloat16()
    run(sa2, torch.ones_like(q), (ramp * torch.ones_like(k)).contiguous(), v, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_level_of_the_first_scores(sa2, d, dtype):
    """Rows whose first 64 scores lie far from 0, all at one side of it, beside rows that lie around it:
    the reference of their exponentials is their own maximum."""
    g = torch.Generator(device="cuda").manual_seed(31)
    q, k, v = tensors(1, 2, 2, 300, 200, d, dtype, seed=31, amp=0.25)
    level = torch.tensor([0.0, -4.0, 5.0, -9.0, 9.0, -30.0, 40.0, -200.0, 150.0], device="cuda")
    rows = level[torch.randint(0, len(level), (300,), generator=g, device="cuda")]
    q[..., 0], k[..., 0] = rows.to(dtype)[None, None], 1.0
    run(sa2, q, k, v, scale=1.0)
    k[:, :, 64:, 0] = -1.0  # and those behind them at the other side
    run(sa2, q, k, v, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hkv,N", [(2, 2, 300), (6, 2, 300), (14, 2, 40), (6, 2, 5), (2, 2, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_do_not_depend_on_each_other(sa2, d, H, Hkv, N, dtype):
    """The same bits for a row beside rows whose scores leap past every range, and whatever the call before
    left in the parts of a tile that hold no query."""
    q, k, v = tensors(1, H, Hkv, N, 700, d, dtype, seed=33)
    k[:, :, 200:] *= 3
    wild, odd = q.clone(), torch.arange(N, device="cuda") % 7 == 2
    wild[:, :, odd] *= 100
    c = sa2.KvCache8.empty(1, Hkv, 700, d, "cuda")
    kl = torch.tensor([700], dtype=torch.int32, device="cuda")
    sa2.cache8_append(c, k, v, torch.zeros_like(kl))
    for f in (lambda x: sa2.cross_attn_fwd(x, k, v), lambda x: sa2.cache8_attn(x, c, kl)):
        o, lse = f(q)
        for other in (wild, torch.full_like(q, math.nan)):
            o2, lse2 = f(other)
            if other is wild:
                assert torch.equal(o2[:, :, ~odd], o[:, :, ~odd]) and torch.equal(lse2[:, :, ~odd], lse[:, :, ~odd])
            o2, lse2 = f(q)
            assert torch.equal(o2, o) and torch.equal(lse2, lse)
    sa2.check_device()


def test_repeated_calls_are_identical(sa2):
    q, k, v = tensors(2, 8, 2, 70, 3000, 128, torch.bfloat16, seed=7)
    o, lse = sa2.cross_attn_fwd(q, k, v)
    for _ in range(20):
        o2, lse2 = sa2.cross_attn_fwd(q, k, v)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    sa2.check_device()


def test_length_out_of_range_is_clamped_and_reported(sa2):
    q, k, v = tensors(3, 2, 2, 64, 100, 64, torch.bfloat16)
    kl = torch.tensor([-3, 101, 50], dtype=torch.int32, device="cuda")
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    assert sa2.device_status() == 7
    assert sa2.device_status() == 0
    check_forward(o, lse, q, k, v, [0, 100, 50])


def test_graph_and_streams(sa2):
    """A call on a side stream, captured with its own workspace, replayed on new inputs."""
    q, k, v = tensors(1, 6, 2, 40, 2500, 128, torch.bfloat16, seed=8)
    kl = torch.tensor([2500], dtype=torch.int32, device="cuda")
    o, lse = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = sa2.cross_attn_fwd(q, k, v, kv_len=kl, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o3, lse3 = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    q2, k2, v2 = tensors(1, 6, 2, 40, 2500, 128, torch.bfloat16, seed=18)
    for dst, src in ((q, q2), (k, k2), (v, v2)):
        dst.copy_(src)
    kl.fill_(1300)
    g.replay()
    sa2.check_device()
    check_forward(o3, lse3, q2, k2, v2, [1300])


def test_refusals(sa2):
    q, k, v = tensors(2, 4, 2, 64, 100, 64, torch.bfloat16)
    bad = [dict(q=q.float(), k=k.float(), v=v.float()), dict(k=k[:, :, :50]), dict(v=v.half()), dict(k=k.cpu()),
           dict(k=k.transpose(2, 3)), dict(kv_len=torch.tensor([1, 2], device="cuda")),
           dict(kv_len=torch.ones(3, dtype=torch.int32, device="cuda")), dict(o=torch.empty_like(q)[:, :, :10]),
           dict(lse=torch.empty((2, 4, 64), device="cuda", dtype=torch.float64)), dict(q=q.cpu(), k=k.cpu(), v=v.cpu())]
    for kw in bad:
        with pytest.raises(ValueError):
            sa2.cross_attn_fwd(**{**dict(q=q, k=k, v=v), **kw})
    with pytest.raises(sa2.Sa2Error):  # three query heads cannot share two key heads
        sa2.cross_attn_fwd(q[:, :3].contiguous(), k, v)
    with pytest.raises(sa2.Sa2Error):  # rows that do not start on 16 bytes
        sa2.cross_attn_fwd(torch.empty((2, 4, 64, 68), device="cuda", dtype=q.dtype)[..., :64], k, v)
    with pytest.raises(sa2.Sa2Error):  # a broadcast batch of keys
        sa2.cross_attn_fwd(q, k[:1].expand(2, -1, -1, -1), v)
    qs = torch.zeros((1, 1, 1, 64), device="cuda", dtype=torch.bfloat16)
    ks = torch.zeros((1, 1, 4000, 64), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(sa2.Sa2Error):  # a workspace too small for the split
        sa2.cross_attn_fwd(qs, ks, ks, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert sa2.device_status() == 0
