"""Cross and cache attention on a stream that the caller names, with nothing that orders it behind the
current stream but the inputs' own readiness: workspaces and outputs that a call makes are no memory that
work of another stream still uses, and tensors may be dropped while the stream still runs."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")
WAIT = 4_000_000  # cycles that the current stream is kept busy for: 2 ms


def calls(m, which, seed):
    """A call of this kind (f(stream) -> its outputs) on inputs of its own."""
    N, M, d = {"split": (40, 6000, 128), "few": (1, 20000, 128), "cache": (40, 6000, 64), "token": (1, 20000, 128),
               "direct": (4000, 300, 64), "backward": (3000, 500, 128), "read": (2, 6000, 128)}[which]
    q, k, v = tensors(1, 8, 4, N, M, d, torch.bfloat16, seed=seed)
    if which in ("cache", "token", "read"):
        c = m.KvCache8.empty(1, 4, M, d, "cuda")
        m.cache8_append(c, k, v, torch.zeros(1, **I32))
        n, first = torch.full((1,), M - 3, **I32), torch.zeros(1, **I32)
        if which == "read":
            return lambda s: m.cache8_read(c, first, 5000, stream=s)
        return lambda s: m.cache8_attn(q, c, n, stream=s)
    if which == "backward":
        o, lse = m.cross_attn_fwd(q, k, v)
        do = torch.randn_like(q)
        return lambda s: m.cross_attn_bwd(q, k, v, o, lse, do, stream=s)
    return lambda s: m.cross_attn_fwd(q, k, v, stream=s)


KINDS = ["split", "few", "cache", "token", "direct", "backward"]


@pytest.mark.parametrize("which", KINDS)
def test_beside_a_call_on_the_current_stream(sa2, which):  # noqa: F811
    """The current stream's call gives its workspace back as it returns, long before its kernels run."""
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


@pytest.mark.parametrize("which", KINDS + ["read"])
def test_outputs_are_no_memory_that_the_current_stream_still_writes(sa2, which):  # noqa: F811
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


@pytest.mark.parametrize("which", ["split", "direct"])
def test_inputs_may_be_dropped(sa2, which):  # noqa: F811
    N, M = (40, 6000) if which == "split" else (4000, 300)
    q, k, v = tensors(1, 8, 4, N, M, 128, torch.bfloat16, seed=5)
    kl = torch.tensor([M - 70], **I32)
    want = sa2.cross_attn_fwd(q, k, v, kv_len=kl)
    side = torch.cuda.Stream()
    for _ in range(3):
        mine = [x.clone() for x in (q, k, v, kl)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(WAIT)
        got = sa2.cross_attn_fwd(*mine[:3], kv_len=mine[3], stream=side)
        mine.clear()
        for x in (q, k, v, kl):  # the same sizes again, on the current stream, which does not wait
            torch.full_like(x, 9)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    sa2.check_device()


def test_a_cache_may_be_dropped(sa2):  # noqa: F811
    q, k, v = tensors(1, 4, 4, 20, 3000, 128, torch.bfloat16, seed=6)
    n, side = torch.full((1,), 3000, **I32), torch.cuda.Stream()

    def cache():
        c = sa2.KvCache8.empty(1, 4, 3000, 128, "cuda")
        sa2.cache8_append(c, k, v, n - 3000)
        return c

    want = sa2.cache8_attn(q, cache(), n)
    for _ in range(3):
        c = cache()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(WAIT)
        got = sa2.cache8_attn(q, c, n, stream=side)
        sizes = [x.shape for x in (c.k, c.v, c.k_scale, c.v_scale)]
        del c
        for s in sizes[:2]:
            torch.zeros(s, dtype=torch.uint8, device="cuda")
        for s in sizes[2:]:
            torch.zeros(s, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    sa2.check_device()


def test_outputs_may_be_dropped_while_they_are_read(sa2):  # noqa: F811
    f, g = calls(sa2, "direct", 7), calls(sa2, "direct", 8)
    want = f(None)[0].float()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        o, lse = f(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(WAIT)
        copy = o.float()  # on the current stream, after the wait
        del o, lse
        g(side)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)
    sa2.check_device()


def test_in_a_graph_and_on_the_default_stream(sa2):  # noqa: F811
    f = calls(sa2, "split", 9)
    want = f(None)
    assert all(torch.equal(x, y) for x, y in zip(f(torch.cuda.default_stream()), want))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = f(side)
        torch.cuda.current_stream().wait_stream(side)
    for x in got:
        x.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    sa2.check_device()


def test_the_current_stream_is_as_it_was(sa2):  # noqa: F811
    f, side = calls(sa2, "few", 10), torch.cuda.Stream()
    torch.cuda.synchronize()
    mine = torch.cuda.Stream()
    with torch.cuda.stream(mine):
        f(side)
        assert torch.cuda.current_stream() == mine
    q, k, v = tensors(1, 2, 2, 3, 70, 64, torch.bfloat16)
    with pytest.raises(ValueError):
        sa2.cross_attn_fwd(q, k, v[:, :1], stream=side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
