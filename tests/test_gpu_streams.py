"""The sparse attention's calls on a stream that the caller names, with nothing that orders it behind the
current stream but the inputs' own readiness: outputs and workspaces are no memory that work of another
stream still uses, and tensors may be dropped while the stream still runs."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cross import sa2, tensors  # noqa: E402,F401

pytestmark = pytest.mark.gpu
WAIT = 4_000_000  # cycles that a stream is kept busy for: 2 ms


def calls(m, which, seed):
    """A call of this kind (f(stream) -> its defined outputs) on inputs of its own."""
    q, k, v = tensors(1, 4, 4, 1500, 1500, 64, torch.bfloat16, seed=seed)
    bm = m.build_mask(q, k, 0.2, 0.5)
    if which == "mask":
        def f(s):
            x = m.build_mask(q, k, 0.2, 0.5, stream=s)
            return x.row_cnt, x.col_cnt, x.mask
        return f
    o, lse = m.attn_fwd(q, k, v, bm)
    do = torch.randn_like(q)
    return {"forward": lambda s: m.attn_fwd(q, k, v, bm, stream=s),
            "backward": lambda s: m.attn_bwd(q, k, v, o, lse, do, bm, stream=s),
            "loss": lambda s: m.vd_loss(o, v, stream=s)}[which]


@pytest.mark.parametrize("which", ["mask", "forward", "backward", "loss"])
def test_beside_a_call_on_the_current_stream(sa2, which):  # noqa: F811
    mine, other = (calls(sa2, which, s) for s in (1, 2))
    want, theirs = mine(None), other(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(10):
        a = other(None)
        b = mine(side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, theirs)), i
        assert all(torch.equal(x, y) for x, y in zip(b, want)), i
    sa2.check_device()


@pytest.mark.parametrize("which", ["mask", "forward", "backward", "loss"])
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


def test_tensors_may_be_dropped(sa2):  # noqa: F811
    """Inputs and the mask's lists while the named stream runs, outputs while the current one reads them."""
    q, k, v = tensors(1, 4, 4, 1500, 1500, 128, torch.bfloat16, seed=5)
    want = sa2.attn_fwd(q, k, v, sa2.build_mask(q, k, 0.2, 0.5))
    every = sa2.build_mask(q, k, 1.0, 1.0)
    side = torch.cuda.Stream()
    for _ in range(3):
        mine, bm = [x.clone() for x in (q, k, v)], sa2.build_mask(q, k, 0.2, 0.5)
        shapes = [(x.shape, x.dtype) for x in bm.tensors() if x is not None]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(WAIT)
        o, lse = sa2.attn_fwd(*mine, bm, stream=side)
        mine.clear()
        del bm
        for x in (q, k, v):  # the same sizes again, on the current stream, which does not wait
            torch.full_like(x, 9)
        for s, t in shapes:
            torch.zeros(s, dtype=t, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(WAIT)
        copy = o.clone(), lse.clone()  # on the current stream, after the wait
        del o, lse
        sa2.attn_fwd(k, q, v, every, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(copy, want))
    sa2.check_device()
