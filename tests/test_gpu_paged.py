"""The paged cache on the GPU: appended tokens against their places, attention over it against its formula in 64
bits, what pages hold outside the sequences, and lengths, pages and places out of range."""
import copy

import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import HostPages, I32, U, attend, check_one, places, shuffled_table, tokens  # noqa: E402

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    return m


def make(sa2, held, page, Hkv, d, dtype, seed=0, width=None, fill=NAN):
    """A cache whose pages hold `fill` but for the sequences' tokens, and its table."""
    table, pages = shuffled_table(held, page, width=width, seed=seed)
    cache = sa2.PagedCache.empty(pages, Hkv, page, d, "cuda", dtype)
    cache.k.fill_(fill)
    cache.v.fill_(fill)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, m in enumerate(held):
        t = torch.arange(m, device="cuda")
        ids, slot = table[b].long()[t // page], t % page
        for x in (cache.k, cache.v):
            x[ids, :, slot] = torch.randn((m, Hkv, d), generator=g, device="cuda").to(dtype)
    return cache, table


def run(sa2, new, held, page, H, Hkv, d, dtype=torch.bfloat16, causal=True, max_new=None, seed=0, width=None, append=True):
    cache, table = make(sa2, held, page, Hkv, d, dtype, seed, width)
    at = places(new)
    seq, kv_len = torch.tensor(at, **I32), torch.tensor(held, **I32)
    q = tokens(H, at[-1], d, dtype, seed + 1)
    host = HostPages(cache, table)
    if append:
        k, v = (tokens(Hkv, at[-1], d, dtype, seed + 2 + i) for i in range(2))
        before = [x.clone() for x in (cache.k, cache.v)]
        sa2.paged_append(cache, k, v, seq, kv_len, table)
        sa2.check_device()
        for b, (n, m) in enumerate(zip(new, held)):
            for x, y in zip(host.tokens(b, m), (k, v)):
                assert torch.equal(x[:, m - n:], y[:, at[b]:at[b + 1]])
        # nothing else has changed
        for x, y, z in zip((cache.k, cache.v), before, (k, v)):
            for b, (n, m) in enumerate(zip(new, held)):
                t = torch.arange(m - n, m, device="cuda")
                y[table[b].long()[t // page], :, t % page] = z[:, at[b]:at[b + 1]].transpose(0, 1)
            assert torch.equal(x.nan_to_num(9.0), y.nan_to_num(9.0))
    o, lse = sa2.paged_attn(q, cache, seq, kv_len, table, causal=causal, max_new=max_new)
    sa2.check_device()
    for b, (n, m) in enumerate(zip(new, held)):
        if n:
            w = slice(at[b], at[b + 1])
            check_one(o[:, w], lse[:, w], q[:, w], *host.tokens(b, m), causal, None, f"sequence {b}")
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)], ids=["64-fp16", "128-bf16"])
@pytest.mark.parametrize("new,held", [([5, 1, 0, 77], [400, 300, 50, 77]), ([200], [1000]), ([1, 1, 1], [1, 129, 640]),
                                      ([130, 3], [130, 515])], ids=str)
def test_pages(sa2, page, d, dtype, new, held):
    run(sa2, new, held, page, 4, 2, d, dtype)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (7, 1), (40, 8), (12, 12), (64, 1), (16, 1), (17, 1)])
@pytest.mark.parametrize("max_new", [None, 1])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens(sa2, H, Hkv, max_new, d):
    """One token for each sequence, over short and long caches; one has only that token, one no new token."""
    run(sa2, [1, 1, 1, 0, 1], [1, 2000, 333, 17, 3001], 64, H, Hkv, d, max_new=max_new, seed=H)


@pytest.mark.parametrize("new", [[2, 2], [3, 1], [4, 4], [16, 7], [8, 0]], ids=str)
@pytest.mark.parametrize("H,Hkv,d,dtype", [(4, 4, 128, torch.bfloat16), (8, 2, 64, torch.float16), (6, 2, 128, torch.float16), (5, 1, 64, torch.bfloat16)])
@pytest.mark.parametrize("causal", [True, False])
def test_few_tokens(sa2, new, H, Hkv, d, dtype, causal):
    """Both sides of the kernel for few rows."""
    run(sa2, new, [1500, 40], 32, H, Hkv, d, dtype, causal, max_new=max(new))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,held", [([300], [5000]), ([64, 500], [3000, 2500]), ([2000], [2000])], ids=str)
def test_chunks_over_long_caches(sa2, causal, new, held):
    run(sa2, new, held, 64, 8, 4, 128, causal=causal)
    run(sa2, new, held, 128, 6, 2, 64, torch.float16, causal)


def test_mixed_batch(sa2):
    run(sa2, [1] * 20 + [300] + [1] * 20, [(37 * b) % 1500 + 1 for b in range(20)] + [900] + [(91 * b) % 1500 + 1 for b in range(20)],
        32, 8, 2, 64)


def test_many_heads_and_sequences(sa2):
    """Whole segments from the counter."""
    run(sa2, [40] * 50, [100 + 7 * b for b in range(50)], 16, 64, 64, 64)


def test_wide_tables(sa2):
    """Room for far more pages than a sequence has: the columns behind are not read."""
    run(sa2, [3, 1], [100, 30], 16, 4, 4, 128, width=4000)
    run(sa2, [3, 1], [100, 30], 16, 4, 4, 128, width=4000, max_new=3)


def test_table_rows_apart_and_strided_pages(sa2):
    """A table with strided rows, pages that lie token by token, K and V in one tensor."""
    held, page, Hkv, d = [200, 77], 32, 2, 64
    table, pages = shuffled_table(held, page, seed=3)
    wide = torch.full((2, 64), -7, **I32)
    wide[:, :table.shape[1]] = table
    both = torch.full((pages, 2, page, Hkv, d), NAN, device="cuda", dtype=torch.bfloat16)
    cache = sa2.PagedCache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
    seq, kv_len = torch.tensor([0, 200, 277], **I32), torch.tensor(held, **I32)
    q, k, v = (tokens(h, 277, d, torch.bfloat16, i) for i, h in enumerate((4, 2, 2)))
    t = wide[:, :table.shape[1]]
    assert t.stride(0) == 64
    sa2.paged_append(cache, k, v, seq, kv_len, t)
    o, lse = sa2.paged_attn(q, cache, seq, kv_len, t)
    sa2.check_device()
    for b, w in enumerate((slice(0, 200), slice(200, 277))):
        check_one(o[:, w], lse[:, w], q[:, w], k[:, w], v[:, w])


def test_pages_shared_by_sequences(sa2):
    """A common beginning in the same pages: read by both."""
    page = 16
    cache = sa2.PagedCache.empty(6, 2, page, 64, "cuda")
    k, v = (tokens(2, 48, 64, torch.bfloat16, i) for i in range(2))
    one = torch.tensor([[4, 0, 2]], **I32)
    sa2.paged_append(cache, k, v, torch.tensor([0, 48], **I32), torch.tensor([48], **I32), one)
    table = torch.tensor([[4, 0, 5], [4, 0, 1]], **I32)
    k2, v2, q = (tokens(h, 3, 64, torch.bfloat16, 5 + i) for i, h in enumerate((2, 2, 4)))
    seq, kv_len = torch.tensor([0, 2, 3], **I32), torch.tensor([34, 33], **I32)
    sa2.paged_append(cache, k2, v2, seq, kv_len, table)
    o, lse = sa2.paged_attn(q, cache, seq, kv_len, table)
    sa2.check_device()
    for w in (slice(0, 2), slice(2, 3)):
        check_one(o[:, w], lse[:, w], q[:, w], torch.cat((k[:, :32], k2[:, w]), 1), torch.cat((v[:, :32], v2[:, w]), 1))


@pytest.mark.parametrize("max_new", [None, 2])
def test_lengths_out_of_range(sa2, max_new):
    """Reported; the sequence has no keys then, the others theirs."""
    held = [40, 40, 40]
    cache, table = make(sa2, held, 16, 2, 64, torch.bfloat16)
    q, k, v = (tokens(h, 6, 64, torch.bfloat16, i) for i, h in enumerate((4, 2, 2)))
    seq = torch.tensor([0, 2, 4, 6], **I32)
    for bad in (1, 0, -5, 49, 2**31 - 1, -2**31):
        kv_len = torch.tensor([40, bad, 40], **I32)
        before = cache.k.clone()
        sa2.paged_append(cache, k, v, seq, kv_len, table)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        ids = table[1].long()
        assert torch.equal(cache.k[ids].nan_to_num(5.0), before[ids].nan_to_num(5.0))
        o, lse = sa2.paged_attn(q, cache, seq, kv_len, table, max_new=max_new)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        assert not o[:, 2:4].any() and bool((lse[:, 2:4] == float("-inf")).all())
        for b in (0, 2):
            w = slice(2 * b, 2 * b + 2)
            check_one(o[:, w], lse[:, w], q[:, w], *HostPages(cache, table).tokens(b, 40))


@pytest.mark.parametrize("max_new", [None, 2])
@pytest.mark.parametrize("page", [16, 128])
def test_pages_out_of_range(sa2, max_new, page):
    """Reported; such a page reads as zeros and is not written."""
    held = [3 * page, 40]
    cache, table = make(sa2, held, page, 2, 64, torch.bfloat16)
    q, k, v = (tokens(h, 4, 64, torch.bfloat16, i) for i, h in enumerate((4, 2, 2)))
    seq, kv_len = torch.tensor([0, 2, 4], **I32), torch.tensor(held, **I32)
    good = HostPages(cache, table.clone())
    for bad in (-1, cache.shape[0], 2**31 - 1, -2**31):
        t = table.clone()
        t[0, 1] = bad
        o, lse = sa2.paged_attn(q, cache, seq, kv_len, t, max_new=max_new)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        kk, vv = (x.clone() for x in good.tokens(0, 3 * page))
        kk[:, page:2 * page] = 0
        vv[:, page:2 * page] = 0
        check_one(o[:, :2], lse[:, :2], q[:, :2], kk, vv)
        check_one(o[:, 2:], lse[:, 2:], q[:, 2:], *good.tokens(1, 40))
        t = table.clone()
        t[0, 2] = bad
        before = cache.k.clone()
        sa2.paged_append(cache, k, v, seq, kv_len, t)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        same = cache.k.clone()
        at = torch.arange(38, 40, device="cuda")
        same[table[1].long()[at // page], :, at % page] = before[table[1].long()[at // page], :, at % page]
        assert torch.equal(same.nan_to_num(5.0), before.nan_to_num(5.0))


@pytest.mark.parametrize("max_new", [None, 1])
def test_places_out_of_order(sa2, max_new):
    held = [40, 40]
    cache, table = make(sa2, held, 16, 2, 64, torch.bfloat16)
    q = tokens(4, 2, 64, torch.bfloat16, 0)
    kv_len = torch.tensor(held, **I32)
    for bad in ([0, 2, 1], [-1, 1, 2], [0, 1, 3], [2, 1, 2], [0, 2**31 - 1, 2]):
        o, lse = torch.full_like(q, 3.0), torch.full((4, 2), 3.0, device="cuda")
        sa2.paged_attn(q, cache, torch.tensor(bad, **I32), kv_len, table, max_new=max_new, o=o, lse=lse)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        assert bool((o == 3).all()) and bool((lse == 3).all())


def test_more_new_tokens_than_said(sa2):
    held = [40, 40]
    cache, table = make(sa2, held, 16, 4, 64, torch.bfloat16)
    q = tokens(4, 4, 64, torch.bfloat16, 0)
    sa2.paged_attn(q, cache, torch.tensor([0, 1, 4], **I32), torch.tensor(held, **I32), table, max_new=1)
    with pytest.raises(sa2.Sa2Error, match="bounds"):
        sa2.check_device()


@pytest.mark.parametrize("max_new", [None, 1])
def test_outside_the_sequences(sa2, max_new):
    held = [70, 20]
    cache, table = make(sa2, held, 32, 2, 128, torch.bfloat16)
    q = tokens(8, 9, 128, torch.bfloat16, 0)
    q[:, [0, 1, 2, 5, 6, 7, 8]] = NAN
    o, lse = torch.full_like(q, 7.0), torch.full((8, 9), 7.0, device="cuda")
    sa2.paged_attn(q, cache, torch.tensor([3, 4, 5], **I32), torch.tensor(held, **I32), table, max_new=max_new, o=o, lse=lse)
    sa2.check_device()
    for b in range(2):
        w = slice(3 + b, 4 + b)
        check_one(o[:, w], lse[:, w], q[:, w], *HostPages(cache, table).tokens(b, held[b]))
    for x in (o, lse):
        assert bool((x[:, :3] == 7).all()) and bool((x[:, 5:] == 7).all())


def test_offsets_beyond_32_bits(sa2):
    """Pages of a cache of more than 2^32 elements."""
    page, Hkv, d = 64, 16, 128
    pages = 2**32 // (page * Hkv * d) + 40
    cache = sa2.PagedCache.empty(pages, Hkv, page, d, "cuda")
    ids = [pages - 1, 0, pages - 3, pages // 2, 5]
    table = torch.tensor([ids], **I32)
    n = 5 * page - 3
    k, v = (tokens(Hkv, n, d, torch.bfloat16, i) for i in range(2))
    seq, kv_len = torch.tensor([0, n], **I32), torch.tensor([n], **I32)
    sa2.paged_append(cache, k, v, seq, kv_len, table)
    q = tokens(Hkv, n, d, torch.bfloat16, 3)
    o, lse = sa2.paged_attn(q, cache, seq, kv_len, table)
    one, l1 = sa2.paged_attn(q[:, n - 1:], cache, torch.tensor([0, 1], **I32), kv_len, table, max_new=1)
    sa2.check_device()
    check_one(o, lse, q, k, v)
    check_one(one, l1, q[:, n - 1:], k, v)


def test_no_new_tokens(sa2):
    cache, table = make(sa2, [40], 16, 2, 64, torch.bfloat16)
    seq, kv_len = torch.tensor([0, 0], **I32), torch.tensor([40], **I32)
    q, k, v = (tokens(2, 0, 64, torch.bfloat16, i) for i in range(3))
    sa2.paged_append(cache, k, v, seq, kv_len, table)
    o, lse = sa2.paged_attn(q, cache, seq, kv_len, table)
    assert o.shape == (2, 0, 64) and lse.shape == (2, 0)
    assert sa2.packed_attn_fwd(q, k, v, seq)[0].shape == (2, 0, 64)
    sa2.check_device()


def test_refusals(sa2):
    cache, table = make(sa2, [40, 20], 16, 2, 64, torch.bfloat16)
    seq, kv_len = torch.tensor([0, 1, 2], **I32), torch.tensor([40, 20], **I32)
    q, k, v = (tokens(h, 2, 64, torch.bfloat16, i) for i, h in enumerate((4, 2, 2)))
    good = dict(q=q, cache=cache, seq=seq, kv_len=kv_len, table=table)
    for bad in (dict(q=q.half()), dict(q=q[..., :32]), dict(q=q[:3]), dict(q=q[None]), dict(seq=seq.long()), dict(seq=seq[:2].contiguous()),
                dict(seq=seq.cpu()), dict(kv_len=None), dict(kv_len=kv_len.float()), dict(table=table.long()), dict(table=table[:1]),
                dict(table=table.t()), dict(max_new=0), dict(max_new="x"), dict(lse=torch.empty((4, 2), device="cuda", dtype=torch.bfloat16)),
                dict(o=q[:, :1]), dict(ws=torch.empty(4, device="cuda")), dict(scale=float("nan"))):
        with pytest.raises((ValueError, sa2.Sa2Error)):
            sa2.paged_attn(**{**good, **bad})
    good = dict(cache=cache, k=k, v=v, seq=seq, kv_len=kv_len, table=table)
    for bad in (dict(k=k.half()), dict(v=v[:, :1]), dict(k=k[:1]), dict(kv_len=kv_len[:1].contiguous()), dict(kv_len=None), dict(table=table.cpu())):
        with pytest.raises(ValueError):
            sa2.paged_append(**{**good, **bad})
    for shape in ((4, 2, 24, 64), (4, 2, 8, 64), (4, 2, 0, 64)):
        with pytest.raises(ValueError, match="power of two"):
            sa2.PagedCache.empty(*shape, "cuda")
    with pytest.raises(ValueError):
        sa2.PagedCache(cache.k, cache.v.half())
    with pytest.raises(ValueError):
        sa2.PagedCache(cache.k, cache.v[:3])
    moved = sa2.PagedCache(cache.k.clone(), cache.v.clone())
    moved.k.data = torch.zeros_like(moved.k)
    with pytest.raises(ValueError, match="moved"):
        sa2.paged_attn(q, moved, seq, kv_len, table)
    other = copy.deepcopy(cache)
    assert type(other) is sa2.PagedCache and other.k.data_ptr() != cache.k.data_ptr()
    sa2.paged_append(other, k, v, seq, kv_len, table)
    sa2.check_device()


@pytest.mark.parametrize("H,Hkv,d", [(24, 12, 64), (8, 8, 128), (5, 1, 128)])
@pytest.mark.parametrize("held", ["short", "uneven", "one long"])
def test_many_single_tokens(sa2, held, H, Hkv, d):
    """More segments than SMs: short ones are taken whole, several by each CTA, others cut into runs, where a run may end
    before a segment's first block; some sequences have no new token, two or three have two."""
    B = 75
    lens = {"short": [3 + 41 * b % 250 for b in range(B)], "uneven": [2 + 197 * b % 1400 for b in range(B)],
            "one long": [20 + b if b != 50 else 20000 for b in range(B)]}[held]
    new = [0 if b % 9 == 4 else 2 if b % 31 == 7 else 1 for b in range(B)]
    run(sa2, new, lens, 32, H, Hkv, d, max_new=2, seed=H)


@pytest.mark.parametrize("H,Hkv,d,dtype", [(12, 12, 128, torch.bfloat16), (40, 8, 128, torch.float16), (16, 2, 64, torch.bfloat16), (32, 4, 64, torch.float16)])
def test_single_tokens_are_as_exact_as_their_type(sa2, H, Hkv, d, dtype):
    """P counts in two parts, so that what is left of its rounding is u^2 of its value (in fp16 2^-25 of the row's largest):
    beside it O has its own rounding, the scores' error ds, and 2^-19 for the exponentials and sums in 32 bits."""
    new, held, page = [1, 1, 1], [512, 3, 2500], 32
    cache, table = make(sa2, held, page, Hkv, d, dtype, seed=H)
    q = tokens(H, 3, d, dtype, H + 1)
    o, _ = sa2.paged_attn(q, cache, torch.tensor(places(new), **I32), torch.tensor(held, **I32), table, max_new=1)
    sa2.check_device()
    u, host = U[dtype], HostPages(cache, table)
    for b, m in enumerate(held):
        k, v = host.tokens(b, m)
        ro, _, a, ds = attend(q[:, b:b + 1], k, v)
        bound = u * ro.abs() * (1 + 2.0**-6) + (u * u + 2 * ds[..., None] + 2.0**-19) * a
        if dtype == torch.float16:
            bound = bound + m * 2.0**-25 * float(v.abs().max()) + 2.0**-25
        err = (o[:, b:b + 1].double() - ro).abs()
        assert bool((err <= bound).all()), f"sequence {b}: {float((err / bound).max()):.3f} of the bound"
