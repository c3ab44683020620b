"""The gradient of attention within packed sequences on the GPU against its formula in 64 bits and against
differences."""
import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import I32, attend, check_gradients, places, tokens  # noqa: E402

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    return m


def run(sa2, lens, H, Hkv, d, causal=True, seed=0, scale=None, norm=True):
    at = places(lens)
    T = at[-1]
    q, k, v, do = (tokens(h, T, d, BF16, seed + i) for i, h in enumerate((H, Hkv, Hkv, H)))
    seq = torch.tensor(at, **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq, causal=causal, scale=scale)
    got = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq, causal=causal, scale=scale)
    sa2.check_device()
    for x, y in zip(got, (q, k, v)):
        assert x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype
    check_gradients(got, q, k, v, do, at, causal, scale, norm)


# (The 2-norm's bound supposes sums of many terms: of sequences of a few tokens single roundings decide.)
@pytest.mark.parametrize("lens", [[1], [2], [1, 1, 1, 1], [16, 0, 15], [64], [65]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_short(sa2, lens, d):
    run(sa2, lens, 4, 2, d, norm=False)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_a_single_key_has_no_gradient(sa2, causal, d):
    """The weight of a row's only key is 1 whatever its score: dQ of a token alone (where causal, of a sequence's first
    one) is 0 to the bit, so is dK of a token alone, and dV is dO, summed over the heads that share it."""
    lens = [1, 1, 5, 1, 140]
    at = places(lens)
    q, k, v, do = (tokens(h, at[-1], d, BF16, i) for i, h in enumerate((4, 2, 2, 4)))
    seq = torch.tensor(at, **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq, causal=causal)
    dq, dk, dv = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq, causal=causal)
    sa2.check_device()
    alone = [0, 1, 7]
    assert not dq[:, alone].any() and not dk[:, alone].any() and bool(dq[:, 3].any()) and bool(dk[:, 2].any())
    assert bool(dq[:, [2, 8]].any()) != causal
    both = do[:, alone].float().view(2, 2, 3, d).sum(1)
    assert float((dv[:, alone].float() - both).abs().max()) <= 2.0**-8 * float(both.abs().max())
    check_gradients((dq, dk, dv), q, k, v, do, at, causal, norm=False)


@pytest.mark.parametrize("lens", [[127], [128], [129], [255, 0, 257], [300, 0, 177, 513], [700]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(sa2, lens, d, causal):
    run(sa2, lens, 4, 2, d, causal)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 1), (7, 7), (12, 4), (64, 1), (40, 8), (10, 2), (33, 3)])
@pytest.mark.parametrize("causal", [True, False])
def test_heads(sa2, H, Hkv, causal):
    run(sa2, [130, 1, 333, 0, 64], H, Hkv, 128, causal, seed=H, norm=False)
    run(sa2, [211, 97], H, Hkv, 64, causal, seed=H + 1)


@pytest.mark.parametrize("lens", [[3000], [2049, 1, 1500], [4097]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(2, 1), (2, 2)])
def test_parts_of_key_blocks(sa2, lens, d, H, Hkv):
    """Few key blocks: the query tiles of each are cut into parts."""
    run(sa2, lens, H, Hkv, d, norm=False)


def test_many_items(sa2):
    """More items than SMs for both kernels, in sections of heads."""
    run(sa2, [700] * 9 + [0, 3, 1200], 32, 16, 128, norm=False)
    run(sa2, [300] * 20, 16, 16, 64)
    run(sa2, [(7 * b) % 5 * 11 for b in range(333)], 4, 4, 64, norm=False)


@pytest.mark.parametrize("first,behind", [(0, 50), (3, 0), (17, 131)])
@pytest.mark.parametrize("lens", [[200, 60], [5, 0, 1], [2000]], ids=str)
@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 4), (128, 3, 1)])
def test_outside_the_sequences(sa2, first, behind, lens, d, H, Hkv):
    """Tokens of no sequence: their inputs count for nothing, their gradients stay as they were."""
    at = places(lens, first)
    T = at[-1] + behind
    q, k, v, do = (tokens(h, T, d, BF16, i) for i, h in enumerate((H, Hkv, Hkv, H)))
    for x in (q, k, v, do):
        x[:, :first] = float("nan")
        x[:, at[-1]:] = float("nan")
    seq = torch.tensor(at, **I32)
    o, lse = torch.full_like(q, float("nan")), torch.full((H, T), float("nan"), device="cuda")
    sa2.packed_attn_fwd(q, k, v, seq, o=o, lse=lse)
    grads = [torch.full_like(x, 7.0) for x in (q, k, v)]
    sa2.packed_attn_bwd(q, k, v, o, lse, do, seq, dq=grads[0], dk=grads[1], dv=grads[2])
    sa2.check_device()
    check_gradients(grads, q, k, v, do, at, norm=False)
    for x in grads:
        assert bool((x[:, :first] == 7).all()) and bool((x[:, at[-1]:] == 7).all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 128])
def test_neighbours_do_not_reach_each_other(sa2, causal, d):
    """NaN and infinities in one sequence's inputs and dO stay there."""
    lens = [70, 130, 45]
    at = places(lens)
    q, k, v, do = (tokens(2, at[-1], d, BF16, i) for i in range(4))
    for i, x in enumerate((q, k, v, do)):
        x[:, 70:200] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
    seq = torch.tensor(at, **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq, causal=causal)
    got = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq, causal=causal)
    sa2.check_device()
    for w in (slice(0, 70), slice(200, 245)):
        n = w.stop - w.start
        check_gradients([x[:, w] for x in got], *(x[:, w] for x in (q, k, v, do)), [0, n], causal)


def test_masked_scores_that_overflow(sa2):
    """Scores behind the diagonal far above the row's own: exp of them is infinite, and counts for nothing."""
    n = 200
    for d in (64, 128):
        q, k, v, do = (tokens(1, n, d, BF16, i) for i in range(4))
        k[:, 100:] *= 100
        q[:, 100:] *= 0.01
        seq = torch.tensor([0, n], **I32)
        o, lse = sa2.packed_attn_fwd(q, k, v, seq)
        got = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq)
        sa2.check_device()
        check_gradients(got, q, k, v, do, [0, n], norm=False)


def test_scales_and_strides(sa2):
    for scale in (1e-3, 0.5):
        run(sa2, [200, 130], 2, 2, 64, scale=scale, norm=False)
        run(sa2, [200, 130], 2, 2, 128, scale=scale, norm=False)
    T, H, d = 170, 4, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    qkv = torch.randn((T, 3, H, d), generator=g, device="cuda").bfloat16()
    q, k, v = qkv.permute(1, 2, 0, 3).unbind(0)
    do = torch.randn((H, T, d + 8), generator=g, device="cuda").bfloat16()[:, :, :d]
    grads = torch.empty((T, 3, H, d), device="cuda", dtype=BF16)
    dq, dk, dv = grads.permute(1, 2, 0, 3).unbind(0)
    seq = torch.tensor([0, 99, T], **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq)
    got = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq, dq=dq, dk=dk, dv=dv)
    sa2.check_device()
    assert got[0] is dq and got[1] is dk and got[2] is dv
    check_gradients(got, q, k, v, do, [0, 99, T])


def test_against_differences(sa2):
    """d loss / d x along a direction, loss = sum O * dO in 64 bits: within the sums of what the kernel's bounds
    allow (gradients to 2 u of their norm, tests/cross_util.py), the difference's own error being h^2."""
    at = places([90, 40])
    q, k, v, do = (tokens(2, at[-1], 64, BF16, i) for i in range(4))
    seq = torch.tensor(at, **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq)
    grads = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq)
    sa2.check_device()

    def loss(x):
        return sum((attend(*(t[:, a:b] for t in x))[0] * do[:, a:b].double()).sum() for a, b in zip(at, at[1:]))

    x = [t.double() for t in (q, k, v)]
    h = 2.0**-12
    for i in range(3):
        e = tokens(2, at[-1], 64, torch.float32, 9 + i).double()
        up, down = ([t + s * h * e if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        want = float((loss(up) - loss(down)) / (2 * h))
        got = float((grads[i].double() * e).sum())
        assert abs(got - want) <= 2 * 2.0**-8 * float(grads[i].double().norm() * e.norm()) + h


def test_repeated_calls_give_the_same_bits(sa2):
    """Counted items and parts, on one workspace that earlier calls have used."""
    for lens, H, Hkv, d in (([900] * 8, 32, 16, 128), ([3000, 200], 2, 1, 64)):
        T = sum(lens)
        at = torch.tensor(places(lens), **I32)
        q, k, v, do = (tokens(h, T, d, BF16, i) for i, h in enumerate((H, Hkv, Hkv, H)))
        o, lse = sa2.packed_attn_fwd(q, k, v, at)
        ws = torch.full((256 << 20,), 255, dtype=torch.uint8, device="cuda")
        first = sa2.packed_attn_bwd(q, k, v, o, lse, do, at, ws=ws)
        for _ in range(4):
            again = sa2.packed_attn_bwd(q, k, v, o, lse, do, at, ws=ws)
            assert all(torch.equal(a, b) for a, b in zip(first, again))
    sa2.check_device()


def test_places_out_of_order_are_reported(sa2):
    T = 300
    q, k, v, do = (tokens(2, T, 64, BF16, i) for i in range(4))
    lse = torch.zeros((2, T), device="cuda")
    for seq in ([0, 200, 100], [-1, 100, 300], [0, 100, 301], [5, 4, 300], [0, 2**31 - 1, 300], [-2**31, 0, 300]):
        grads = [torch.full_like(x, 3.0) for x in (q, k, v)]
        sa2.packed_attn_bwd(q, k, v, q, lse, do, torch.tensor(seq, **I32), dq=grads[0], dk=grads[1], dv=grads[2])
        with pytest.raises(sa2.Sa2Error, match="bounds"):
            sa2.check_device()
        assert all(bool((x == 3).all()) for x in grads)


def test_refusals(sa2):
    q, k, v, do = (tokens(h, 10, 64, BF16, i) for i, h in enumerate((4, 2, 2, 4)))
    seq = torch.tensor([0, 10], **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq)
    good = dict(q=q, k=k, v=v, o=o, lse=lse, do=do, seq=seq)
    with pytest.raises(sa2.Sa2Error, match="unsupported"):
        sa2.packed_attn_bwd(*(x.half() for x in (q, k, v, o)), lse, do.half(), seq)
    for bad in (dict(do=do[:, :5]), dict(do=do.half()), dict(lse=lse.double()), dict(lse=lse[:2]), dict(dk=q), dict(seq=seq[:1]),
                dict(o=None), dict(k=k[:, :5]), dict(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(q=q[None])):
        with pytest.raises((ValueError, sa2.Sa2Error)):
            sa2.packed_attn_bwd(**{**good, **bad})
    sa2.check_device()


@pytest.mark.parametrize("lens,H,Hkv", [([152], 32, 2), ([1000], 24, 1), ([129, 40, 900], 16, 1), ([260], 64, 1)], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_more_parts_than_tiles(sa2, lens, H, Hkv, d):
    """Key blocks cut into as many parts as the longest sequences have tiles for: the last blocks have fewer tiles."""
    run(sa2, lens, H, Hkv, d, norm=False)
