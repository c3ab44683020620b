"""Plain 64-bit forms of attention within packed sequences, its gradient, attention over a paged cache and rotary
positions, with the error bounds that the tests of the CUDA kernels use.  Nothing here is shared with the library.

The bounds of O, LSE and the gradients are those of tests/cross_util.py, whose derivation does not depend on which
keys a row has: per element, u |x| for the output's rounding and, of the terms that it sums up, u for each rounding of
P or dS and 2 ds or 4 ds for the scores' error ds <= d 2^-23 sum |q k|.
"""
import math

import torch

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
I32 = dict(dtype=torch.int32, device="cuda")


def places(lens, first=0):
    """seq of sequences of these lengths, the first from token `first` on."""
    at = [first]
    for n in lens:
        at.append(at[-1] + n)
    return at


def tokens(H, T, d, dtype, seed, scale=1.0, token_major=True):
    """[H, T, d], as a view of a projection's [T, H, d] where token_major."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (T, H, d) if token_major else (H, T, d)
    x = (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)
    return x.transpose(0, 1) if token_major else x


def allowed(n, m, causal, device):
    """[n, m]: the keys of each of the last n of m tokens."""
    if not causal:
        return torch.ones((n, m), dtype=torch.bool, device=device)
    return torch.arange(m, device=device) <= torch.arange(m - n, m, device=device)[:, None]


def attend(q, k, v, causal=True, scale=None):
    """One sequence: q [H, n, d], the last n of the m tokens of k, v [Hkv, m, d].  O, LSE, A = sum p |v|, ds."""
    H, n, d = q.shape
    G, m = H // k.shape[0], k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    keep = allowed(n, m, causal, q.device)
    o, lse, a, ds = [], [], [], []
    for h in range(H):
        qq, kk, vv = q[h].double(), k[h // G].double(), v[h // G].double()
        s = (qq @ kk.T * scale).masked_fill(~keep, -math.inf)
        ds.append((qq.abs() @ kk.abs().T * keep).amax(1) * scale * d * 2.0**-23)
        lse.append(torch.logsumexp(s, 1))
        p = torch.exp(s - lse[-1][:, None])
        o.append(p @ vv)
        a.append(p @ vv.abs())
    return [torch.stack(x) for x in (o, lse, a, ds)]


def check_one(o, lse, q, k, v, causal=True, scale=None, what=""):
    """Asserts one sequence's O and LSE."""
    ro, rl, a, ds = attend(q, k, v, causal, scale)
    u = U[q.dtype]
    bound = u * ro.abs() * (1 + 2.0**-6) + (u + 2 * ds[..., None] + 2.0**-19) * a + 1e-30
    if q.dtype == torch.float16:  # P below 2^-14 of the row's reference, outputs below 2^-14
        bound = bound + k.shape[1] * 2.0**-25 * float(v.abs().max()) + 2.0**-25
    err = (o.double() - ro).abs()
    assert bool((err <= bound).all()), f"{what} O: {float((err / bound).nan_to_num(math.inf).max()):.3f} of the bound"
    el, bl = (lse.double() - rl).abs(), ds + 2.0**-19 * (rl.abs() + 1)
    assert bool((el <= bl).all()), f"{what} LSE: {float((el / bl).nan_to_num(math.inf).max()):.3f} of the bound"


def check_packed(o, lse, q, k, v, at, causal=True, scale=None):
    for b in range(len(at) - 1):
        w = slice(at[b], at[b + 1])
        if at[b + 1] > at[b]:
            check_one(o[:, w], lse[:, w], q[:, w], k[:, w], v[:, w], causal, scale, f"sequence {b}")


def gradients(q, k, v, do, causal=True, scale=None):
    """One sequence attending to itself: dQ, dK, dV in 64 bits, and of each the sum of the magnitudes it adds up."""
    H, n, d = q.shape
    G = H // k.shape[0]
    scale = scale or 1.0 / math.sqrt(d)
    keep = allowed(n, n, causal, q.device)
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)  # noqa: E731
    dq, dk, dv, aq, ak, av = z(q), z(k), z(v), z(q), z(k), z(v)
    for h in range(H):
        g = h // G
        qq, kk, vv, dd = q[h].double(), k[g].double(), v[g].double(), do[h].double()
        p = torch.softmax((qq @ kk.T * scale).masked_fill(~keep, -math.inf), 1)
        dp = dd @ vv.T
        ds = p * (dp - (p * dp).sum(1, keepdim=True))
        dq[h] = ds @ kk * scale
        dk[g] += ds.T @ qq * scale
        dv[g] += p.T @ dd
        ap = dd.abs() @ vv.abs().T
        da = p * (ap + (p * ap).sum(1, keepdim=True))
        aq[h] = da @ kk.abs() * scale
        ak[g] += da.T @ qq.abs() * scale
        av[g] += p.T @ dd.abs()
    return (dq, dk, dv), (aq, ak, av)


def check_gradients(got, q, k, v, do, at, causal=True, scale=None, norm=True):
    for b in range(len(at) - 1):
        w = slice(at[b], at[b + 1])
        if at[b + 1] == at[b]:
            continue
        x = [t[:, w] for t in (q, k, v, do)]
        want, mags = gradients(*x, causal, scale)
        ds = float(attend(*x[:3], causal, scale)[3].max())
        u = U[q.dtype]
        for name, g, r, a, roundings in zip(("dq", "dk", "dv"), got, want, mags, (2, 2, 1)):
            e = (g[:, w].double() - r).abs()
            bound = u * r.abs() * (1 + 2.0**-6) + (roundings * u + 4 * ds + 2.0**-16) * a + 1e-30
            assert bool((e <= bound).all()), f"sequence {b} {name}: {float((e / bound).nan_to_num(math.inf).max()):.3f} of the bound"
            if norm and float(r.norm()):
                rel = float((g[:, w].double() - r).norm() / r.norm())
                assert rel <= 2 * u, f"sequence {b} {name}: relative error {rel:.2e}"


class HostPages:
    """A paged cache by its definition: a Python list of tokens for each sequence, and where the pages have them."""

    def __init__(self, cache, table):
        self.cache, self.table, self.page = cache, table, cache.shape[2]

    def tokens(self, b, m):
        """K, V of the first m tokens of sequence b: [Hkv, m, d]."""
        t = torch.arange(m, device="cuda")
        ids, slot = self.table[b].long()[t // self.page], t % self.page
        return [x[ids, :, slot].transpose(0, 1) for x in (self.cache.k, self.cache.v)]


def shuffled_table(held, page, spare=2, width=None, seed=0):
    """A table [B, width] for sequences that hold (or will hold) so many tokens, pages in no order, and their count."""
    per = [-(-n // page) for n in held]
    width = width or max(max(per), 1)
    g = torch.Generator().manual_seed(seed)
    order = torch.randperm(sum(per) + spare, generator=g).tolist()
    table, at = torch.full((len(held), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table.cuda(), sum(per) + spare


def turned(x, pos, freq, axis, layout, gain=1.0, inverse=False):
    """Rotary positions in 64 bits: x [B, H, N, d], pos [axes, B, N]."""
    y = x.double().clone()
    f = torch.tensor(freq, dtype=torch.float64, device=x.device)
    t = torch.stack([pos[a].double() * w for w, a in zip(f, axis)], -1)[:, None]
    c, s = torch.cos(t) * gain, torch.sin(t) * gain * (-1 if inverse else 1)
    n = len(freq)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if layout == "interleaved" else (slice(0, n), slice(n, 2 * n))
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y
