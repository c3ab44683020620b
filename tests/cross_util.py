"""Plain 64-bit forms of cross attention, its gradient and the 8-bit cache, with the error bounds that
the tests of the CUDA kernels use.  Nothing here is shared with the library.

Bounds (u = eps / 2 is the relative error of one rounding, per type):

O     the output's rounding, u |O|; P's rounding, u A with A = sum p |v|; the scores' error ds, which
      changes p by at most 2 ds relatively; the exponentials and sums in fp32, 2^-19 A at most.  ds: a
      sum of d products in fp32 is off by at most d 2^-23 sum |q k| (any order of summation).
      fp16 P: below 2^-14 of the row's reference it is held to within 2^-25 absolutely, which over M
      keys adds M 2^-25 max|v| (the row's largest p is at least 1 in that scale; with a cache the
      reference includes V's scale, so that max|v| is 448 times the largest scale).
LSE   ds + 2^-19 (|LSE| + 1).

dV    the output's rounding, u |dV|, and (u + 4 ds + 2^-16) sum p |dO|: P's rounding, what the scores
      and the LSE (each by ds) change p by, and fp32 sums.
dQ,   u |dQ| and (2 u + 4 ds + 2^-16) sum |dS||k| with |dS| taken by its terms, p (|dO||v| + sum p
dK    |dO||v|): dS is rounded (u) and D = dO . O is made from the rounded O (u).
In the 2-norm the roundings are independent and each is u / sqrt(3) of its term on average, so that
with random inputs, where no sum cancels, the whole gradient is within sqrt(3) u / sqrt(3) = u of
its norm; the tests ask for 2 u.
"""
import math

import torch

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}
BLOCK, E_MIN, E_MAX = 64, -100, 119


def lengths(kv_len, B, M):
    return [M] * B if kv_len is None else [int(x) for x in kv_len]


def attention(q, k, v, lens, scale=None):
    """O, LSE, A = sum p |v| and ds (bound of a row's score error) in 64 bits; k, v any dtype."""
    B, H, N, d = q.shape
    G = H // k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    o = torch.zeros((B, H, N, d), dtype=torch.float64, device=q.device)
    a = torch.zeros_like(o)
    lse = torch.full((B, H, N), -math.inf, dtype=torch.float64, device=q.device)
    ds = torch.zeros((B, H, N), dtype=torch.float64, device=q.device)
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        for h in range(H):
            kk, vv, qq = k[b, h // G, :n].double(), v[b, h // G, :n].double(), q[b, h].double()
            s = qq @ kk.T * scale
            ds[b, h] = (qq.abs() @ kk.abs().T).amax(1) * scale * d * 2.0**-23
            lse[b, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[b, h][:, None])
            o[b, h] = p @ vv
            a[b, h] = p @ vv.abs()
    return o, lse, a, ds


def gradients(q, k, v, do, lens, scale=None):
    """dQ, dK, dV in 64 bits, and for each the sum of the magnitudes that it adds up."""
    B, H, N, d = q.shape
    Hkv, G = k.shape[1], H // k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    z = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=q.device)  # noqa: E731
    dq, dk, dv, aq, ak, av = z(q), z(k), z(v), z(q), z(k), z(v)
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        for h in range(H):
            g = h // G
            kk, vv, qq, dd = k[b, g, :n].double(), v[b, g, :n].double(), q[b, h].double(), do[b, h].double()
            p = torch.softmax(qq @ kk.T * scale, 1)
            dp = dd @ vv.T
            D = (p * dp).sum(1, keepdim=True)
            ds = p * (dp - D)
            dq[b, h] = ds @ kk * scale
            dk[b, g, :n] += ds.T @ qq * scale
            dv[b, g, :n] += p.T @ dd
            # magnitudes: |dP| and |D| by their terms
            ap = dd.abs() @ vv.abs().T
            da = p * (ap + (p * ap).sum(1, keepdim=True))
            aq[b, h] = da @ kk.abs() * scale
            ak[b, g, :n] += da.T @ qq.abs() * scale
            av[b, g, :n] += p.T @ dd.abs()
    return (dq, dk, dv), (aq, ak, av)


def check_forward(o, lse, q, k, v, lens, scale=None, p_type=None, v_max=None):
    """Asserts O and LSE of a call against the bounds above; p_type: the type P is rounded to."""
    ro, rl, a, ds = attention(q, k, v, lens, scale)
    p_type = p_type or q.dtype
    tiny = 0.0
    if p_type == torch.float16:
        v_max = v_max if v_max is not None else max([float(v[b, :, :n].abs().max()) for b, n in enumerate(lens) if n] or [0.0])
        tiny = k.shape[2] * 2.0**-25 * v_max
    bound = U[q.dtype] * ro.abs() * (1 + 2.0**-6) + (U[p_type] + 2 * ds[..., None] + 2.0**-19) * a + tiny + 1e-30
    if q.dtype == torch.float16:
        bound = bound + 2.0**-25  # spacing of fp16 outputs below 2^-14
    err = (o.double() - ro).abs()
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, f"O: {worst:.3f} of the bound, max error {float(err.max()):.3e}"
    empty = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty), "LSE of rows without keys"
    el = torch.where(empty, 0.0, (lse.double() - torch.where(empty, 0.0, rl)).abs().nan_to_num(math.inf))
    el = torch.where(empty, 0.0, el)
    bl = ds + 2.0**-19 * (torch.where(empty, 0.0, rl).abs() + 1)
    assert float((el / bl).max()) <= 1.0, f"LSE: {float((el / bl).max()):.3f} of the bound"
    return worst


def check_gradients(got, q, k, v, do, lens, scale=None, norm=True):
    want, mags = gradients(q, k, v, do, lens, scale)
    ds = float(attention(q, k, v, lens, scale)[3].max())
    u = U[q.dtype]
    for name, g, w, a, roundings in zip(("dq", "dk", "dv"), got, want, mags, (2, 2, 1)):
        assert g.shape == w.shape and g.dtype == q.dtype
        bound = u * w.abs() * (1 + 2.0**-6) + (roundings * u + 4 * ds + 2.0**-16) * a
        err = (g.double() - w).abs()
        over = torch.where(err > 0, err / bound.clamp(min=1e-300), 0.0)
        assert float(over.max()) <= 1.0, f"{name}: {float(over.max()):.3f} of the bound, max error {float(err.max()):.3e}"
        if norm and float(w.norm()):
            rel = float((g.double() - w).norm() / w.norm())
            assert rel <= 2 * u, f"{name}: relative error {rel:.2e}"


# ------------------------------------------------------------------------------ 8-bit cache


def round_e4m3(x):
    """Nearest e4m3 value (64 bits), ties to even, largest magnitude 448."""
    x = x.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(x / step) * step


def exponent(amax):
    """Least e with amax <= 448 * 2^e, within the cache's limits."""
    if amax == 0:
        return E_MIN
    e = math.floor(math.log2(amax / 448)) - 1
    while amax > 448 * 2.0**e:
        e += 1
    return min(max(e, E_MIN), E_MAX)


class HostCache:
    """The cache by its definition: values in 64 bits, one sequence, head and block at a time."""

    def __init__(self, B, H, C, d):
        self.x = torch.zeros((B, H, C, d), dtype=torch.float64)  # e4m3 values
        self.e = torch.zeros((B, H, -(-C // BLOCK)), dtype=torch.int64)

    def append(self, x, pos, counts):
        B, H, n, d = x.shape
        x = x.double().cpu()
        for b in range(B):
            p, m = pos[b], counts[b]
            for j in range(p // BLOCK, (p + m - 1) // BLOCK + 1 if m else 0):
                lo, hi = max(p, j * BLOCK), min(p + m, (j + 1) * BLOCK)
                for h in range(H):
                    new = x[b, h, lo - p:hi - p]
                    e = exponent(float(new.abs().max()))
                    if j * BLOCK < p:
                        was = int(self.e[b, h, j])
                        e = max(e, was)
                        old = self.x[b, h, j * BLOCK:p]
                        self.x[b, h, j * BLOCK:p] = round_e4m3(old * 2.0 ** (was - e))
                    self.x[b, h, lo:hi] = round_e4m3(new * 2.0**-e)
                    self.e[b, h, j] = e

    def values(self):
        C = self.x.shape[2]
        return self.x * torch.exp2(self.e.double()).repeat_interleave(BLOCK, 2)[:, :, :C, None]


def cache_values(x8, scale):
    """The values (64 bits) of device tensors in the cache's form."""
    C = x8.shape[2]
    return x8.view(torch.float8_e4m3fn).float().double() * scale.double().repeat_interleave(BLOCK, 2)[:, :, :C, None]
