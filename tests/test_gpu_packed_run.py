"""Rotary positions, packed attention and the paged cache as they are used together; calls on several streams, in
graphs, that fail, and that are repeated."""
import pytest

torch = pytest.importorskip("torch")

from tests.packed_util import (HostPages, I32, U, attend, check_gradients, check_one, check_packed, places,  # noqa: E402
                               shuffled_table, tokens, turned)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TIMEOUT = 6
WAIT = 4_000_000  # cycles that the current stream is kept busy for: 2 ms


@pytest.fixture(scope="module")
def sa2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_sparse_attention_sa2_gb300 as m
    m.load_library()
    m.device_status()
    yield m
    m.debug_set_wait_limit(0, 0)


def positions(lens, first=None):
    return torch.cat([torch.arange(n) + (first[b] if first else 0) for b, n in enumerate(lens)]).to(**I32)


def test_a_training_step(sa2):
    """Queries and keys turned, attention, and the way back to the gradients of what was turned: each part against
    its formula on what it was given, and the whole against autograd in 64 bits (2 roundings of each of q', k', o, the
    gradients of q', k' and their turned ones: 8 u of the norm)."""
    lens, H, Hkv, d = [130, 0, 77, 301], 6, 2, 64
    at = places(lens)
    T = at[-1]
    q, k, v, do = (tokens(h, T, d, BF16, i) for i, h in enumerate((H, Hkv, Hkv, H)))
    r = sa2.Rotary(d, sa2.rotary_frequencies(48), layout="half")
    pos, seq = positions(lens), torch.tensor(at, **I32)
    q1, k1 = sa2.rotary(r, pos, q, k)
    o, lse = sa2.packed_attn_fwd(q1, k1, v, seq)
    dq1, dk1, dv = sa2.packed_attn_bwd(q1, k1, v, o, lse, do, seq)
    dq, dk = sa2.rotary(r, pos, dq1, dk1, inverse=True)
    sa2.check_device()
    check_packed(o, lse, q1, k1, v, at)
    check_gradients((dq1, dk1, dv), q1, k1, v, do, at)
    x = [t.double().requires_grad_() for t in (q, k, v)]
    turn = lambda t: turned(t[None], pos[None, None], r.frequencies, [0] * 24, "half")[0]  # noqa: E731
    xq, xk = turn(x[0]), turn(x[1])
    loss = 0.0
    for a, b in zip(at, at[1:]):
        if b > a:
            s = torch.einsum("hnd,hmd->hnm", xq[:, a:b], xk[:, a:b].repeat_interleave(3, 0)) / d**0.5
            p = torch.softmax(s + torch.full((b - a, b - a), float("-inf"), device="cuda", dtype=torch.float64).triu(1), 2)
            loss = loss + ((p @ x[2][:, a:b].repeat_interleave(3, 0)) * do[:, a:b].double()).sum()
    for got, want in zip((dq, dk, dv), torch.autograd.grad(loss, x)):
        assert float((got.double() - want).norm() / want.norm()) <= 8 * U[BF16]


@pytest.mark.parametrize("page", [16, 128])
def test_prompts_then_tokens(sa2, page):
    """Prompts of a batch attended to at once and put into pages, then chunks and single tokens: every step's output is
    that of the whole sequences' attention."""
    H, Hkv, d, B = 8, 2, 64, 4
    steps = [[150, 33, 1, 260], [1, 1, 1, 1], [1, 20, 1, 0], [1, 1, 64, 1], [1, 1, 1, 1]]
    total = [sum(s[b] for s in steps) for b in range(B)]
    table, pages = shuffled_table(total, page)
    cache = sa2.PagedCache.empty(pages, Hkv, page, d, "cuda")
    r = sa2.Rotary(d, sa2.rotary_frequencies(d))
    held = [0] * B
    whole = [[], []]
    for i, new in enumerate(steps):
        T = sum(new)
        q, k, v = (tokens(h, T, d, BF16, 10 * i + j) for j, h in enumerate((H, Hkv, Hkv)))
        q, k = sa2.rotary(r, positions(new, held), q, k)
        at = places(new)
        held = [m + n for m, n in zip(held, new)]
        seq, kv_len = torch.tensor(at, **I32), torch.tensor(held, **I32)
        sa2.paged_append(cache, k, v, seq, kv_len, table)
        o, lse = sa2.paged_attn(q, cache, seq, kv_len, table, max_new=max(new) if i % 2 else None)
        sa2.check_device()
        host = HostPages(cache, table)
        for b, n in enumerate(new):
            w = slice(at[b], at[b + 1])
            if n:
                check_one(o[:, w], lse[:, w], q[:, w], *host.tokens(b, held[b]), what=f"step {i} sequence {b}")
        if i == 0:  # nothing before it: the same as the prompts' own attention
            o2, lse2 = sa2.packed_attn_fwd(q, k, v, seq)
            sa2.check_device()
            check_packed(o2, lse2, q, k, v, at)
        for j, x in enumerate((k, v)):
            whole[j].append([x[:, at[b]:at[b + 1]] for b in range(B)])
    for b in range(B):
        for x, kept in zip(host.tokens(b, held[b]), whole):
            assert torch.equal(x, torch.cat([s[b] for s in kept], 1))


def test_frames_of_a_clip(sa2):
    """Frame by frame: the new frame's tokens see each other whole and all before (causal off), positions on three axes."""
    frames, h, w, H, d = 3, 6, 9, 4, 128
    n = h * w
    f = [x for c in (44, 42, 42) for x in sa2.rotary_frequencies(c)]
    r = sa2.Rotary(d, f, axes=[22, 21, 21])
    table, pages = shuffled_table([frames * n], 16)
    cache = sa2.PagedCache.empty(pages, H, 16, d, "cuda")
    i = torch.arange(n)
    for t in range(frames):
        q, k, v = (tokens(H, n, d, BF16, 3 * t + j) for j in range(3))
        pos = torch.stack([torch.full((n,), t), i // w, i % w]).to(**I32)
        q1, k1 = sa2.rotary(r, pos, q, k)
        seq, kv_len = torch.tensor([0, n], **I32), torch.tensor([(t + 1) * n], **I32)
        sa2.paged_append(cache, k1, v, seq, kv_len, table)
        o, lse = sa2.paged_attn(q1, cache, seq, kv_len, table, causal=False)
        sa2.check_device()
        check_one(o, lse, q1, *HostPages(cache, table).tokens(0, (t + 1) * n), causal=False)


def calls(m, which, seed):
    """A call of this kind (f(stream) -> its outputs) on inputs of its own."""
    H, Hkv, lens, d = {"split": (2, 2, [5000, 300], 128), "direct": (16, 8, [700] * 6, 64), "backward": (8, 4, [1500, 200], 128),
                       "parts": (2, 1, [3000], 64), "token": (8, 4, [1] * 5, 128), "chunk": (8, 2, [64, 1, 1], 64), "mixed": (8, 4, [300, 1, 1, 2], 64),
                       "append": (4, 4, [77, 3], 64), "rotary": (4, 4, [2000], 64)}[which]
    at = places(lens)
    T = at[-1]
    q, k, v, do = (tokens(h, T, d, BF16, seed + i) for i, h in enumerate((H, Hkv, Hkv, H)))
    seq = torch.tensor(at, **I32)
    if which in ("backward", "parts"):
        o, lse = m.packed_attn_fwd(q, k, v, seq)
        return lambda s: m.packed_attn_bwd(q, k, v, o, lse, do, seq, stream=s)
    if which == "rotary":
        r, pos = m.Rotary(d, m.rotary_frequencies(d)), torch.arange(T, **I32)
        return lambda s: m.rotary(r, pos, q, k, stream=s)
    if which in ("token", "chunk", "mixed", "append"):
        held = [3000 + 100 * b for b in range(len(lens))]
        table, pages = shuffled_table(held, 64, seed=seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        cache = m.PagedCache(*(torch.randn((pages, Hkv, 64, d), generator=g, device="cuda").bfloat16() for _ in range(2)))
        kv_len = torch.tensor(held, **I32)
        if which == "append":
            def f(s):
                m.paged_append(cache, k, v, seq, kv_len, table, stream=s)
                return m.paged_attn(q, cache, seq, kv_len, table, stream=s)
            return f
        return lambda s: m.paged_attn(q, cache, seq, kv_len, table, max_new=max(lens), stream=s)
    return lambda s: m.packed_attn_fwd(q, k, v, seq, stream=s)


KINDS = ["split", "direct", "backward", "parts", "token", "chunk", "mixed", "append", "rotary"]


@pytest.mark.parametrize("which", KINDS)
def test_beside_a_call_on_the_current_stream(sa2, which):
    """Two calls at once, each with a workspace of its own, the current stream's given back as the call returns."""
    mine, other = (calls(sa2, which, s) for s in (1, 2))
    want, theirs = mine(None), other(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(20):
        if i % 2:
            torch.cuda._sleep(WAIT // 40)
        a = other(None)
        b = mine(side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, theirs)), i
        assert all(torch.equal(x, y) for x, y in zip(b, want)), i
    sa2.check_device()


@pytest.mark.parametrize("which", KINDS)
def test_outputs_are_no_memory_that_the_current_stream_still_writes(sa2, which):
    f = calls(sa2, which, 3)
    want = f(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        used = [torch.empty_like(x) for x in want for _ in range(3)]
        torch.cuda._sleep(WAIT)
        for x in used:
            x.fill_(7)  # runs after the wait
        del used, x
        got = f(side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    sa2.check_device()


def test_inputs_may_be_dropped(sa2):
    lens, side = [2000, 300], torch.cuda.Stream()
    q, k, v = (tokens(4, 2300, 64, BF16, i) for i in range(3))
    seq = torch.tensor(places(lens), **I32)
    want = sa2.packed_attn_fwd(q, k, v, seq)
    for _ in range(3):
        mine = [x.clone() for x in (q, k, v, seq)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(WAIT)
        got = sa2.packed_attn_fwd(*mine, stream=side)
        mine.clear()
        for x in (q, k, v, seq):  # the same sizes again, on the current stream, which does not wait
            torch.full_like(x, 9)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    sa2.check_device()


@pytest.mark.parametrize("which", KINDS)
def test_each_kernel_waits_for_what_the_one_before_wrote(sa2, which):
    """A chain on one stream, each call's inputs written just before it: kernels begin early, but read late."""
    f = calls(sa2, which, 5)
    want = f(None)
    torch.cuda.synchronize()
    for _ in range(30):
        got = f(None)
        again = f(None)
        total = [x.float().sum() for x in got]  # reads what the calls wrote, while more calls follow
        f(None)
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and all(torch.equal(x, y) for x, y in zip(again, want))
        assert all(torch.equal(x, y.float().sum()) for x, y in zip(total, want))
    sa2.check_device()


def test_inputs_written_just_before(sa2):
    """q is written by a kernel that the attention follows at once, every time with other values."""
    lens, T = [200, 56], 256
    seq = torch.tensor(places(lens), **I32)
    base, k, v = (tokens(4, T, 64, BF16, i) for i in range(3))
    want = [sa2.packed_attn_fwd((base.float() * (1 + i)).bfloat16(), k, v, seq)[0] for i in range(4)]
    torch.cuda.synchronize()
    q = torch.empty_like(base)
    scaled = [(base.float() * (1 + i)).bfloat16() for i in range(4)]
    for i in range(40):
        q.copy_(scaled[i % 4])
        o, _ = sa2.packed_attn_fwd(q, k, v, seq)
        q.fill_(0)  # and overwritten just behind
        assert torch.equal(o, want[i % 4])


@pytest.mark.parametrize("which", KINDS)
def test_captured_and_replayed(sa2, which):
    """Two graphs with workspaces of their own that are replayed at once, beside an eager call."""
    f, g = calls(sa2, which, 7), calls(sa2, which, 8)
    want = [f(None), g(None)]
    graphs, outs = [], []
    for h in (f, g):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(h(None))
    side = torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            for x in o:
                x.fill_(0)
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        eager = f(None)
        torch.cuda.synchronize()
        for got, w in zip(outs + [eager], want + [want[0]]):
            assert all(torch.equal(x, y) for x, y in zip(got, w))
    sa2.check_device()


def test_a_graph_with_other_lengths_and_pages(sa2):
    """A token step captured once serves batches of other lengths, places and tables of the same sizes."""
    H, Hkv, d, page, B = 8, 2, 128, 32, 3
    table = torch.zeros((B, 40), **I32)
    cache = sa2.PagedCache.empty(130, Hkv, page, d, "cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for x in (cache.k, cache.v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    q, k, v = (tokens(h, 4, d, BF16, i) for i, h in enumerate((H, Hkv, Hkv)))
    seq, kv_len = torch.zeros(B + 1, **I32), torch.ones(B, **I32)

    def step():
        sa2.paged_append(cache, k, v, seq, kv_len, table)
        return sa2.paged_attn(q, cache, seq, kv_len, table, max_new=2)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    sa2.device_status()
    for i, (new, held) in enumerate((([2, 1, 1], [1280, 3, 700]), ([1, 1, 1], [64, 65, 1]), ([0, 2, 2], [0, 1000, 1279]), ([1, 0, 2], [33, 5, 2]))):
        order = torch.randperm(130, generator=torch.Generator().manual_seed(i))[:120].reshape(3, 40)
        table.copy_(order)
        seq.copy_(torch.tensor(places(new)))
        kv_len.copy_(torch.tensor(held))
        graph.replay()
        sa2.check_device()
        host, at = HostPages(cache, table), places(new)
        for b in range(B):
            w = slice(at[b], at[b + 1])
            if new[b]:
                check_one(o[:, w], lse[:, w], q[:, w], *host.tokens(b, held[b]))


def test_calls_keep_no_memory(sa2):
    fs = [calls(sa2, which, 9) for which in KINDS]
    for f in fs:
        f(None)
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    for _ in range(20):
        for f in fs:
            f(None)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == held


@pytest.mark.parametrize("which", ["split", "direct", "chunk", "backward", "parts"])
def test_expired_wait_reports_timeout_and_the_context_survives(sa2, which):
    f = calls(sa2, which, 11)
    want = f(None)
    sa2.check_device()
    sa2.debug_set_wait_limit(2_000_000, 200_000_000)
    try:
        f(None)
        status = sa2.device_status()
    finally:
        sa2.debug_set_wait_limit(0, 0)
    assert status == TIMEOUT
    got = f(None)
    sa2.check_device()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_many_sequences(sa2):
    """Thousands of sequences, most of them of one token or none, in every call."""
    B, H, d = 3333, 2, 64
    lens = [1 if b % 3 else 0 for b in range(B)]
    lens[700], lens[3000] = 300, 40
    at = places(lens)
    T = at[-1]
    q, k, v, do = (tokens(H, T, d, BF16, i) for i in range(4))
    seq = torch.tensor(at, **I32)
    o, lse = sa2.packed_attn_fwd(q, k, v, seq)
    grads = sa2.packed_attn_bwd(q, k, v, o, lse, do, seq)
    held = [n + b % 50 if n else 0 for b, n in enumerate(lens)]
    table, pages = shuffled_table(held, 16)
    cache = sa2.PagedCache.empty(pages, H, 16, d, "cuda")
    cache.k.normal_(), cache.v.normal_()
    kv_len = torch.tensor(held, **I32)
    sa2.paged_append(cache, k, v, seq, kv_len, table)
    o2, lse2 = sa2.paged_attn(q, cache, seq, kv_len, table)
    sa2.check_device()
    one = [b for b in range(B) if lens[b] == 1]
    w = torch.tensor([at[b] for b in one], device="cuda")
    assert torch.equal(o[:, w], v[:, w])  # a token alone: its own value
    s = (q[:, w].double() * k[:, w].double()).sum(2) / 8
    assert float((lse[:, w].double() - s).abs().max()) <= 1e-4  # d 2^-23 sum |q k| / 8 is 4e-5 for sums of 41, 2^-19 (|LSE| + 1) 1e-5
    assert torch.equal(grads[2][:, w], do[:, w])
    host = HostPages(cache, table)
    for b in [700, 3000] + one[::97]:
        x = slice(at[b], at[b + 1])
        if lens[b] > 1:
            check_one(o[:, x], lse[:, x], q[:, x], k[:, x], v[:, x])
            check_gradients([t[:, x] for t in grads], *(t[:, x] for t in (q, k, v, do)), [0, lens[b]], norm=False)
        check_one(o2[:, x], lse2[:, x], q[:, x], *host.tokens(b, held[b]))
