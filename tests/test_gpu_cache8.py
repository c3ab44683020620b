"""The 8-bit key/value cache (sa2_cache8_append / _read / _attn) against plain 64-bit forms
(tests/cross_util.py): the held values exactly, attention within derived bounds."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_util import HostCache, cache_values, check_forward  # noqa: E402

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    return m


def random_cache(sa2, B, H, C, d, seed=0, spread=3):
    """A cache whose blocks' scales differ by factors of up to 2^(2 spread)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = sa2.KvCache8.empty(B, H, C, d, "cuda")
    pos = torch.zeros(B, **I32)
    nb = -(-C // 64)
    for _ in range(2):
        kv = []
        for _ in range(2):
            mag = torch.exp2(torch.randint(-spread, spread + 1, (B, H, nb), generator=g, device="cuda").float())
            x = torch.randn((B, H, C, d), generator=g, device="cuda") * mag.repeat_interleave(64, 2)[:, :, :C, None]
            kv.append(x.bfloat16())
    sa2.cache8_append(c, kv[0] * 0.5, kv[1], pos)
    return c


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_append_in_pieces(sa2, d, dtype):
    """Pieces of many lengths, growing and shrinking magnitudes, ragged counts: every held byte and
    scale as the definition gives them; what lies behind is left as it was."""
    B, H, C = 3, 2, 500
    c = sa2.KvCache8.empty(B, H, C, d, "cuda")
    for t in (c.k, c.v):
        t.view(torch.uint8).fill_(0x7F)
    c.k_scale.fill_(math.nan), c.v_scale.fill_(math.nan)
    host = [HostCache(B, H, C, d) for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(1)
    pos = [0, 5, 63]
    for b in range(B):  # positions before the first one hold zeros under scale 1
        for t in (c.k, c.v):
            t.view(torch.uint8)[b, :, :pos[b]] = 0
    c.k_scale[:, :, 0] = c.v_scale[:, :, 0] = 1.0
    for step, (n, amp) in enumerate([(1, 1.0), (1, 8.0), (63, 0.1), (64, 30.0), (65, 1e-3), (2, 900.0), (130, 1e-6), (1, 0.0)]):
        counts = [n, max(0, n - 1 - step % 2), n // 2]
        k, v = ((torch.randn((B, H, n, d), generator=g, device="cuda") * amp * f).to(dtype) for f in (1.0, 3.0))
        args = (torch.tensor(pos, **I32), None if step == 0 else torch.tensor(counts, **I32))
        counts = [n] * B if step == 0 else counts
        sa2.cache8_append(c, k, v, *args)
        for hc, x in zip(host, (k, v)):
            hc.append(x, pos, counts)
        pos = [p + m for p, m in zip(pos, counts)]
        sa2.check_device()
        for hc, x8, sc in ((host[0], c.k, c.k_scale), (host[1], c.v, c.v_scale)):
            want, got = hc.values(), cache_values(x8, sc).cpu()
            for b in range(B):
                assert torch.equal(got[b, :, :pos[b]], want[b, :, :pos[b]]), (step, b)
                assert bool((x8.view(torch.uint8)[b, :, pos[b]:] == 0x7F).all()), "bytes behind the end"
                assert bool(sc[b, :, -(-pos[b] // 64):].isnan().all()) or pos[b] == 0, "scales behind the end"
    first = torch.tensor([0, 3, 60], **I32)
    n = min(pos) - 60
    kk, vv = sa2.cache8_read(c, first, n, dtype=dtype)
    sa2.check_device()
    for hc, x in zip(host, (kk, vv)):
        w = hc.values()
        for b, p in enumerate((0, 3, 60)):
            assert torch.equal(x[b].cpu(), w[b, :, p:p + n].to(dtype))


def test_append_limits(sa2):
    """Zeros, the smallest and largest magnitudes, infinities and NaN."""
    c = sa2.KvCache8.empty(1, 1, 256, 64, "cuda")
    big = torch.finfo(torch.bfloat16).max
    x = torch.zeros((1, 1, 256, 64), device="cuda", dtype=torch.bfloat16)
    x[0, 0, 64:128] = 1e-38
    x[0, 0, 128:192, 0] = 2.0**127
    x[0, 0, 192, 0], x[0, 0, 193, 1], x[0, 0, 194, 2] = big, math.inf, math.nan
    sa2.cache8_append(c, x, x, torch.zeros(1, **I32))
    assert sa2.device_status() == 8
    got = cache_values(c.k, c.k_scale)[0, 0].cpu()
    assert torch.equal(c.k_scale[0, 0].cpu(), torch.tensor([2.0**-100, 2.0**-100, 2.0**119, 2.0**119]))
    assert bool((got[:128] == 0).all()) and bool((got[128:192, 0] == 2.0**127).all())
    most = 448 * 2.0**119
    assert float(got[192, 0]) == most and float(got[193, 1]) == most and math.isnan(float(got[194, 2]))


def test_append_and_read_out_of_range(sa2):
    c = sa2.KvCache8.empty(2, 1, 100, 64, "cuda")
    x = torch.ones((2, 1, 10, 64), device="cuda", dtype=torch.bfloat16)
    guard = c.k.view(torch.uint8)
    guard.fill_(1)
    c.k_scale.fill_(1), c.v_scale.fill_(1)
    sa2.cache8_append(c, x, x, torch.tensor([95, 0], **I32))
    assert sa2.device_status() == 7
    assert torch.equal(cache_values(c.k, c.k_scale)[0, 0, 95:].float(), torch.ones((5, 64), device="cuda"))
    sa2.cache8_append(c, x, x, torch.tensor([-1, 200], **I32), torch.tensor([11, 3], **I32))
    assert sa2.device_status() == 7
    k, _ = sa2.cache8_read(c, torch.tensor([97, -2], **I32), 6)
    assert sa2.device_status() == 7
    assert bool((k[0, 0, 3:] == 0).all()) and bool((k[0, 0, :3] == 1).all()) and bool((k[1, 0, :2] == 0).all())
    sa2.cache8_append(c, x[:, :, :0], x[:, :, :0], torch.zeros(2, **I32))
    assert sa2.device_status() == 0


def attend(sa2, q, c, lens, scale=None):
    kl = torch.tensor(lens, **I32)
    o = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:3], math.nan, dtype=torch.float32, device="cuda")
    for b, n in enumerate(lens):  # behind the end: NaN bytes and NaN scales
        for x8, sc in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x8.view(torch.uint8)[b, :, n:] = 0x7F
            sc[b, :, -(-n // 64):] = math.nan
    sa2.cache8_attn(q, c, kl, scale=scale, o=o, lse=lse)
    sa2.check_device()
    k, v = cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale)
    v_max = 448 * max([float(c.v_scale[b, :, :-(-n // 64)].max()) for b, n in enumerate(lens) if n] or [0.0])
    check_forward(o, lse, q, k, v, lens, scale, p_type=torch.float16, v_max=v_max)
    return o, lse


def queries(B, H, N, d, dtype, seed=0, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((B, N, H, d), generator=g, device="cuda") * amp).to(dtype).transpose(1, 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 3, 17, 128, 200])
@pytest.mark.parametrize("n", [1, 16, 63, 64, 65, 128, 129, 500])
def test_attention_sizes(sa2, N, n, d):
    attend(sa2, queries(2, 4, N, d, torch.bfloat16, seed=N), random_cache(sa2, 2, 2, 512, d, seed=n), [n, max(0, n - 2)])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (7, 1), (16, 1), (20, 1), (64, 1), (5, 5)])
@pytest.mark.parametrize("N", [1, 4, 60])
def test_attention_heads(sa2, H, Hkv, N, dtype):
    attend(sa2, queries(3, H, N, 128, dtype, seed=H), random_cache(sa2, 3, Hkv, 1500, 128, seed=N), [1500, 0, 701])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 300])
def test_attention_long(sa2, N, d):
    attend(sa2, queries(2, 6, N, d, torch.bfloat16), random_cache(sa2, 2, 2, 9000, d), [9000, 4001])


def test_attention_scale_of_rows(sa2):
    """bf16 queries far outside the fp16 range: each row has its own power of two."""
    c = random_cache(sa2, 1, 1, 200, 64)
    q = queries(1, 1, 40, 64, torch.bfloat16, amp=1e-3)
    base = attend(sa2, q, c, [200])
    for f in (2.0**40, 2.0**-60):
        o, lse = sa2.cache8_attn(q * f, c, torch.tensor([200], **I32), scale=0.125 / f)
        sa2.check_device()
        assert torch.equal(o, base[0]) and torch.equal(lse, base[1])


def test_attention_repeats_and_graph(sa2):
    for N in (1, 50):
        c, q = random_cache(sa2, 2, 2, 3000, 128), queries(2, 4, N, 128, torch.bfloat16)
        kl = torch.tensor([3000, 1234], **I32)
        o, lse = sa2.cache8_attn(q, c, kl)
        for _ in range(10):
            o2, lse2 = sa2.cache8_attn(q, c, kl)
            assert torch.equal(o, o2) and torch.equal(lse, lse2)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o3, lse3 = sa2.cache8_attn(q, c, kl)
        q.copy_(queries(2, 4, N, 128, torch.bfloat16, seed=5))
        kl.copy_(torch.tensor([77, 2999], **I32))
        g.replay()
        sa2.check_device()
        k, v = cache_values(c.k, c.k_scale), cache_values(c.v, c.v_scale)
        check_forward(o3, lse3, q, k, v, [77, 2999], p_type=torch.float16, v_max=448 * float(c.v_scale.max()))


def test_streamed_frames(sa2):
    """Frame by frame as it is used: append, attend over all so far; the first frames' values stay."""
    B, H, d, n = 1, 4, 128, 150
    c = sa2.KvCache8.empty(B, H, 1000, d, "cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    kept = []
    pos = torch.zeros(B, **I32)
    for step in range(6):
        k, v = (torch.randn((B, n, H, d), generator=g, device="cuda").bfloat16().transpose(1, 2) for _ in range(2))
        sa2.cache8_append(c, k, v, pos)
        pos += n
        o, lse = sa2.cache8_attn(k, c, pos)
        sa2.check_device()
        total = n * (step + 1)
        rk, rv = sa2.cache8_read(c, torch.zeros(B, **I32), total)
        check_forward(o, lse, k, rk, rv, [total], p_type=torch.float16, v_max=448 * float(c.v_scale[:, :, :-(-total // 64)].max()))
        # the same attention over the values read back
        o2, lse2 = sa2.cross_attn_fwd(k, rk, rv)
        check_forward(o2, lse2, k, rk, rv, [total])
        kept.append((rk, total))
    assert all(torch.allclose(a[:, :, :m].float(), kept[-1][0][:, :, :m].float(), rtol=2.0**-4, atol=0.2) for a, m in kept)


def test_refusals(sa2):
    c = random_cache(sa2, 2, 2, 128, 64)
    q, kl = queries(2, 4, 3, 64, torch.bfloat16), torch.tensor([5, 6], **I32)
    x = torch.zeros((2, 2, 4, 64), device="cuda", dtype=torch.bfloat16)
    for f in (lambda: sa2.cache8_attn(q.float(), c, kl), lambda: sa2.cache8_attn(q, c, None),
              lambda: sa2.cache8_attn(q, c, kl.long()), lambda: sa2.cache8_attn(q[:1], c, kl[:1]),
              lambda: sa2.cache8_append(c, x, x.half(), kl), lambda: sa2.cache8_append(c, x[:, :1], x[:, :1], kl),
              lambda: sa2.cache8_append(c, x, x, kl[:1]), lambda: sa2.cache8_append(c, x, x, None),
              lambda: sa2.cache8_read(c, kl, 4, dtype=torch.float32), lambda: sa2.cache8_read(c, None, 4),
              lambda: sa2.KvCache8(c.k, c.v[:, :, :64], c.k_scale, c.v_scale),
              lambda: sa2.KvCache8(c.k, c.v, c.k_scale[:, :, :1], c.v_scale),
              lambda: sa2.KvCache8(c.k.float(), c.v.float(), c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(sa2.Sa2Error):  # three query heads, two key heads
        sa2.cache8_attn(q[:, :3].contiguous(), c, kl)
    assert sa2.device_status() == 0
