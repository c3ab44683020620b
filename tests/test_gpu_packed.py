"""Attention within packed sequences on the GPU against its formula in 64 bits: types, shared heads, lengths,
strides, what lies outside the sequences, and repeated calls."""
import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import I32, check_one, check_packed, places, tokens  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    return m


def run(sa2, lens, H, Hkv, d, dtype, causal=True, seed=0, scale=None, qscale=1.0):
    at = places(lens)
    T = at[-1]
    q, k, v = (tokens(h, T, d, dtype, seed + i, s) for i, (h, s) in enumerate(((H, qscale), (Hkv, 1.0), (Hkv, 1.0))))
    o, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor(at, **I32), causal=causal, scale=scale)
    sa2.check_device()
    assert o.shape == q.shape and o.dtype == dtype and lse.shape == (H, T) and lse.dtype == torch.float32
    check_packed(o, lse, q, k, v, at, causal, scale)


# one token, a tile's edge, a half block's, a block's, a pair's, and more
LENGTHS = [[1], [2], [16], [63], [64], [65], [127], [128], [129], [255, 1, 0, 257], [0, 0, 5], [1, 1, 1, 1, 1], [300, 0, 77, 513]]


@pytest.mark.parametrize("lens", LENGTHS, ids=str)
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)], ids=["64-fp16", "128-bf16"])
def test_lengths(sa2, lens, d, dtype):
    run(sa2, lens, 4, 2, d, dtype)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 1), (7, 7), (12, 4), (64, 1), (40, 8), (10, 2), (33, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_heads(sa2, H, Hkv, causal):
    run(sa2, [130, 1, 333, 0, 64], H, Hkv, 128, torch.bfloat16, causal, seed=H)
    run(sa2, [211, 97], H, Hkv, 64, torch.bfloat16, causal, seed=H + 1)


@pytest.mark.parametrize("lens", [[3000], [2049, 1, 1500], [1, 4097]], ids=str)
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16)], ids=["64-bf16", "128-fp16"])
@pytest.mark.parametrize("causal", [True, False])
def test_split_keys(sa2, lens, d, dtype, causal):
    """Few heads: the keys of a segment are split over CTAs."""
    run(sa2, lens, 2, 1, d, dtype, causal)


@pytest.mark.parametrize("G", [1, 3, 5, 8])
def test_split_cuts_every_way(sa2, G):
    """Runs that begin and end anywhere in sequences of any length."""
    for i, lens in enumerate(([1100, 1030, 1], [1024, 1025, 1026, 1500], [5000, 3, 900, 2222])):
        run(sa2, lens, 2 * G, 2, 64, torch.bfloat16, seed=i)


@pytest.mark.parametrize("causal", [True, False])
def test_many_items(sa2, causal):
    """More segments than SMs: work comes from the counter, in sections of heads."""
    run(sa2, [700] * 9 + [0, 3, 1200], 32, 16, 128, torch.bfloat16, causal)
    run(sa2, [37] * 100, 16, 16, 64, torch.float16, causal)


def test_many_short_sequences(sa2):
    """More sequences than a warp looks at in one step, empty ones in between."""
    run(sa2, [(7 * b) % 5 * 11 for b in range(333)], 4, 4, 64, torch.bfloat16)
    run(sa2, [1] * 100, 8, 2, 128, torch.float16)


@pytest.mark.parametrize("first,behind", [(0, 50), (3, 0), (17, 131)])
@pytest.mark.parametrize("lens", [[200, 60], [5, 0, 1]], ids=str)
def test_outside_the_sequences(sa2, first, behind, lens):
    """Tokens of no sequence: their inputs count for nothing, their outputs stay as they were."""
    at = places(lens, first)
    T = at[-1] + behind
    q, k, v = (tokens(4, T, 64, torch.bfloat16, i) for i in range(3))
    for x in (q, k, v):
        x[:, :first] = float("nan")
        x[:, at[-1]:] = float("inf")
    o, lse = torch.full_like(q, 7.0), torch.full((4, T), 7.0, device="cuda")
    sa2.packed_attn_fwd(q, k, v, torch.tensor(at, **I32), o=o, lse=lse)
    sa2.check_device()
    check_packed(o, lse, q, k, v, at)
    for x in (o, lse):
        assert bool((x[:, :first] == 7).all()) and bool((x[:, at[-1]:] == 7).all())


@pytest.mark.parametrize("causal", [True, False])
def test_neighbours_do_not_reach_each_other(sa2, causal):
    """NaN and infinities in one sequence stay there."""
    at = places([70, 130, 45])
    q, k, v = (tokens(2, at[-1], 128, torch.bfloat16, i) for i in range(3))
    for i, x in enumerate((q, k, v)):
        x[:, 70:200] = (float("nan"), float("inf"), float("-inf"))[i]
    o, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor(at, **I32), causal=causal)
    sa2.check_device()
    for w in (slice(0, 70), slice(200, 245)):
        check_one(o[:, w], lse[:, w], q[:, w], k[:, w], v[:, w], causal)


def test_masked_keys_count_for_nothing(sa2):
    """Keys of later tokens, NaN and infinite ones too, and large scores behind the diagonal."""
    n = 200
    q, k, v = (tokens(2, n, 64, torch.bfloat16, i) for i in range(3))
    seq = torch.tensor([0, n], **I32)
    k2, v2 = k.clone(), v.clone()
    k2[:, 150:] = float("nan")
    k2[:, 190:] = 1e30
    o1, lse1 = sa2.packed_attn_fwd(q, k, v, seq)
    o2, lse2 = sa2.packed_attn_fwd(q, k2, v2, seq)
    sa2.check_device()
    assert torch.equal(o1[:, :150], o2[:, :150]) and torch.equal(lse1[:, :150], lse2[:, :150])
    # a value reaches tokens up to 127 before it, which share products with it, at most
    v2[:, 199:] = float("nan")
    o3, _ = sa2.packed_attn_fwd(q, k, v2, seq)
    assert torch.equal(o1[:, :72], o3[:, :72])


def test_infinite_keys_are_left_out(sa2):
    n = 100
    q, k, v = (tokens(1, n, 64, torch.bfloat16, i).abs() for i in range(3))
    k[:, 0] = float("-inf")
    k[:, 70] = float("-inf")
    o, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor([0, n], **I32))
    sa2.check_device()
    assert float(lse[0, 0]) == float("-inf") and not o[0, 0].any()
    keep = [i for i in range(n) if i not in (0, 70)]
    check_one(o[:, keep], lse[:, keep], q[:, keep], k[:, keep], v[:, keep])


def test_scores_that_jump(sa2):
    """Scores far above everything before them: references follow, rows of one tile each on their own."""
    n = 700
    for dtype, jump in ((torch.bfloat16, 500.0), (torch.float16, 60.0)):
        q = torch.ones((2, n, 64), device="cuda", dtype=dtype)
        k = torch.zeros((2, n, 64), device="cuda", dtype=dtype)
        v = tokens(2, n, 64, dtype, 3)
        for i, f in ((70, 0.25), (200, 0.5), (330, 1.0), (599, 0.9)):
            k[:, i] = f * jump / 64
        o, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor([0, 100, n], **I32), scale=1.0)
        sa2.check_device()
        check_packed(o, lse, q, k, v, [0, 100, n], scale=1.0)


def test_scales(sa2):
    for scale in (1e-3, 0.5, 3.0):
        run(sa2, [100, 30], 2, 2, 64, torch.bfloat16, scale=scale)


@pytest.mark.parametrize("layout", ["head major", "token major", "wide rows", "one head of many"])
def test_strides(sa2, layout):
    T, H, d = 170, 4, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    if layout == "head major":
        q, k, v = (r(H, T, d) for _ in range(3))
    elif layout == "token major":
        q, k, v = r(T, 3, H, d).permute(1, 2, 0, 3).unbind(0)  # one projection of all three
    elif layout == "wide rows":
        q, k, v = (r(H, T, d + 72)[:, :, 8:8 + d] for _ in range(3))
    else:
        q, k, v = (r(H * 3, T, d)[::3] for _ in range(3))
    at = [0, 99, T]
    o = torch.empty((T, H, d + 8), device="cuda", dtype=torch.bfloat16)[:, :, :d].transpose(0, 1)
    o2, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor(at, **I32), o=o)
    sa2.check_device()
    assert o2 is o
    check_packed(o, lse, q, k, v, at)


def test_repeated_calls_give_the_same_bits(sa2):
    """Direct with the counter, and split, on one workspace that earlier calls have used."""
    for lens, H, Hkv in (([900] * 8, 32, 16), ([3000, 200], 2, 1)):
        at = torch.tensor(places(lens), **I32)
        q, k, v = (tokens(h, sum(lens), 64, torch.bfloat16, i) for i, h in enumerate((H, Hkv, Hkv)))
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
        first = sa2.packed_attn_fwd(q, k, v, at, ws=ws)
        for _ in range(4):
            again = sa2.packed_attn_fwd(q, k, v, at, ws=ws)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    sa2.check_device()


def test_places_out_of_order_are_reported(sa2):
    """Nothing is written then."""
    T = 300
    q, k, v = (tokens(2, T, 64, torch.bfloat16, i) for i in range(3))
    for seq in ([0, 200, 100], [-1, 100, 300], [0, 100, 301], [5, 4, 300], [0, 2**31 - 1, 300], [-2**31, 0, 300]):
        o = torch.full_like(q, 3.0)
        lse = torch.full((2, T), 3.0, device="cuda")
        sa2.packed_attn_fwd(q, k, v, torch.tensor(seq, **I32), o=o, lse=lse)
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        assert bool((o == 3).all()) and bool((lse == 3).all())


@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)], ids=["64-fp16", "128-bf16"])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (6, 1), (33, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_every_place_of_the_last_key(sa2, d, dtype, H, Hkv, causal):
    """Sequences that end at each place within half a block of keys, whose last scores are cut row by row."""
    lens = [64 + n for n in range(0, 64, 7)] + [1, 31, 32, 33, 63, 191, 255]
    at = places(lens)
    q, k, v = (tokens(h, at[-1], d, dtype, i) for i, h in enumerate((H, Hkv, Hkv)))
    o, lse = sa2.packed_attn_fwd(q, k, v, torch.tensor(at, **I32), causal=causal)
    sa2.check_device()
    check_packed(o, lse, q, k, v, at, causal)
