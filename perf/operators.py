"""Cases that measure attention of queries to keys of another length: cross attention with its
gradient, and attention over keys and values that a cache holds in 8 bits.

``run`` computes each operator in plain torch operations (``own = False``) or through this
package's entry points (``own = True``) on the same inputs.  Four kinds of case:

* ``cross``   O, LSE of queries [B, H, N, d] over keys and values [B, Hkv, M, d], key lengths per
              sequence optional;
* ``train``   the same with dQ, dK, dV for a given dO: one training step of the sublayer;
* ``append``  new keys and values into the 8-bit cache behind what it holds, and those tokens
              read back as the values that they are held as;
* ``cached``  O, LSE of queries over the 8-bit cache.

The 8-bit form: e4m3 values and, for each head and block of 64 tokens, one scale, the least power of
two 2^e with amax <= 448 * 2^e (e kept within [-100, 119]).  A block that is extended keeps the
larger of its scale and the one that the new tokens need; when that grows, the tokens that it holds
are rounded again under the new scale.
"""
import math

import torch

own = False

BLOCK = 64
E_MIN, E_MAX = -100, 119


def listed():
    return [
        # text states of 512 tokens read by one layer's video tokens, Wan2.1 1.3B at 480p and 14B at 720p
        dict(name="cross 480p", kind="cross", B=1, H=12, Hkv=12, N=32760, M=512, d=128, type="bf16", lens="full"),
        dict(name="cross 720p", kind="cross", B=1, H=40, Hkv=40, N=75600, M=512, d=128, type="bf16", lens="full"),
        # a small padded batch of prompts, one of them empty: latency counts
        dict(name="cross small", kind="cross", B=4, H=8, Hkv=8, N=256, M=77, d=64, type="fp16", lens="ragged"),
        # few learned queries over the states of a whole clip: the key axis is the long one
        dict(name="cross few queries", kind="cross", B=2, H=24, Hkv=8, N=64, M=32760, d=128, type="bf16", lens="ragged"),
        # a training step of the text cross attention
        dict(name="train 480p", kind="train", B=1, H=12, Hkv=12, N=32760, M=512, d=128, type="bf16", lens="full"),
        # image and text states of odd length, key heads shared, a padded batch
        dict(name="train shared heads", kind="train", B=3, H=24, Hkv=8, N=8190, M=769, d=64, type="bf16", lens="ragged"),
        # one frame's tokens (45 x 80) put behind the frames that the cache holds, in the middle of a block
        dict(name="append frame", kind="append", B=1, Hkv=40, M=75600, n=3600, d=128, type="bf16", lens="odd"),
        # one token for each sequence of a batch
        dict(name="append token", kind="append", B=16, Hkv=8, M=4096, n=1, d=128, type="bf16", lens="ragged"),
        # one query token for each sequence of a batch over long caches
        dict(name="cached token", kind="cached", B=8, H=40, Hkv=40, N=1, M=32760, d=128, type="bf16", lens="ragged"),
        # one token over one prompt: latency counts
        dict(name="cached small", kind="cached", B=1, H=12, Hkv=12, N=1, M=512, d=128, type="bf16", lens="full"),
        # one frame's tokens (30 x 52) over the clip so far at 480p, heads of 64
        dict(name="cached frame 480p", kind="cached", B=1, H=24, Hkv=24, N=1560, M=32760, d=64, type="fp16", lens="odd"),
        # one frame's tokens over a whole clip at 720p
        dict(name="cached frame 720p", kind="cached", B=1, H=40, Hkv=40, N=3600, M=75600, d=128, type="bf16", lens="full"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: every size over its logarithm, costs below the largest listed ones."""
    kind = rng.choice(("cross", "cross", "train", "append", "cached", "cached"))
    d = rng.choice((64, 128))
    hkv, group = rng.choice(((12, 1), (40, 1), (24, 1), (8, 3), (8, 1), (4, 8), (5, 1), (1, 7)))
    B = rng.choice((1, 1, 2, 3, 4, 8))
    lens = rng.choice(("full", "ragged", "odd"))
    if kind == "append":
        M = _log(rng, 512, 75600)
        return dict(kind=kind, B=B, Hkv=hkv, M=M, n=_log(rng, 1, min(M // 2, 4000)), d=d, type=rng.choice(("bf16", "fp16")), lens=lens)
    while True:
        n_hi, m_lo, m_hi = {"cross": (75600, 40, 40000), "train": (40000, 40, 4000), "cached": (4000, 100, 75600)}[kind]
        n_lo = 16 if kind == "train" else 1
        N, M = _log(rng, n_lo, n_hi), _log(rng, m_lo, m_hi)
        if B * hkv * group * N * M <= 40 * 75600 * (512 if kind != "cached" else 3600) / 4:
            break
    ty = "bf16" if kind == "train" else rng.choice(("bf16", "bf16", "fp16"))
    return dict(kind=kind, B=B, H=hkv * group, Hkv=hkv, N=N, M=M, d=d, type=ty, lens=lens)


def _lens(c):
    """Key lengths of a case's sequences (append: the tokens that the cache holds before)."""
    M, B = c["M"] - c.get("n", 0), c["B"]
    if c["lens"] == "full":
        return [M] * B
    if c["lens"] == "odd":
        return [max(1, (M - 1 - 5 * b) | 1) if M > 1 else M for b in range(B)]
    got = [max(1, int(M * (1 - 0.61803 * b % 1))) for b in range(B)]
    if B > 2 and "n" not in c:
        got[1] = 0  # a sequence with nothing to attend to
    return got


def _type(c):
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[c["type"]]


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ty, d = _type(c), c["d"]

    def rnd(*shape, scale=1.0, dtype=ty):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(scale).to(dtype)

    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    s = dict(case=dict(c), lens=lens, kv_len=None if c["lens"] == "full" else lens, type=ty)
    if c["kind"] in ("cross", "train"):
        # projections' outputs are token-major [B, N, H, d]: the operators take them as they lie
        s["q"] = rnd(c["B"], c["N"], c["H"], d).transpose(1, 2)
        kv = rnd(2, c["B"], c["M"], c["Hkv"], d)
        pad = torch.arange(c["M"], device=dev) >= lens[:, None]
        kv.masked_fill_(pad[None, :, :, None, None], float("nan"))  # what lies behind a sequence's end is anything
        s["k"], s["v"] = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
        if c["kind"] == "train":
            s["do"] = rnd(c["B"], c["N"], c["H"], d).transpose(1, 2)
        return s
    # the cache: blocks of different magnitude, as activations of different frames and heads have
    cap = -(-c["M"] // BLOCK) * BLOCK
    nb = cap // BLOCK
    s["cache"] = []
    for _ in range(2):
        x = torch.randn((c["B"], c["Hkv"], nb, BLOCK, d), generator=g, device=dev)
        mag = torch.randint(-1, 2, (c["B"], c["Hkv"], nb, 1, 1), generator=g, device=dev).float()
        x.mul_(torch.exp2(mag))
        e = torch.ceil(torch.log2(x.abs().amax((3, 4), keepdim=True) / 448.0)).clamp_(E_MIN, E_MAX)
        x8 = x.mul_(torch.exp2(-e)).clamp_(-448, 448).to(torch.float8_e4m3fn)
        s["cache"].append((x8.view(c["B"], c["Hkv"], cap, d), torch.exp2(e).view(c["B"], c["Hkv"], nb)))
        del x
    if c["kind"] == "cached":
        s["kv_len"] = lens
        s["q"] = rnd(c["B"], c["N"], c["H"], d).transpose(1, 2)
    else:
        kv = rnd(2, c["B"], c["n"], c["Hkv"], d, scale=1.5)
        s["k"], s["v"] = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
    return s


# ---------------------------------------------------------------- the operators in plain form


def _mask(lens, M):
    return torch.arange(M, device=lens.device) < lens[:, None]


def _heads(x, H):
    """[B, Hkv, M, d] in 32 bits with each key head repeated for the query heads that share it."""
    return x.repeat_interleave(H // x.shape[1], dim=1) if H != x.shape[1] else x


def _attend(q, k, v, lens):
    """O and LSE in 32 bits, and what a gradient needs; rows of a sequence without keys get 0 and -inf."""
    M, scale = k.shape[2], 1.0 / math.sqrt(q.shape[3])
    keep = _mask(lens, M)
    k = torch.where(keep[:, None, :, None], k, 0.0)
    v = torch.where(keep[:, None, :, None], v, 0.0)
    s = torch.matmul(q, k.transpose(2, 3))
    s.mul_(scale).masked_fill_(~keep[:, None, None, :], float("-inf"))
    m = s.amax(3, keepdim=True)
    m = torch.where(torch.isinf(m), 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(3, keepdim=True)
    p.div_(torch.where(l > 0, l, 1.0))
    o = torch.matmul(p, v)
    return o, (m + torch.log(l)).squeeze(3), p, k, v, scale


def _shared(x, hkv):
    """Sums the gradient of a shared key head over its query heads."""
    B, H, M, d = x.shape
    return x if H == hkv else x.view(B, hkv, H // hkv, M, d).sum(2)


def _plain_cross(s):
    c, ty = s["case"], s["type"]
    q, k, v = s["q"].float(), _heads(s["k"].float(), c["H"]), _heads(s["v"].float(), c["H"])
    o, lse, p, k, v, scale = _attend(q, k, v, s["lens"])
    if c["kind"] == "cross":
        return {"o": o.to(ty), "lse": lse}
    do = s["do"].float()
    dv = torch.matmul(p.transpose(2, 3), do)
    ds = torch.matmul(do, v.transpose(2, 3))
    ds.sub_((do * o).sum(3, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(scale)
    return {"o": o.to(ty), "lse": lse, "dq": dq.to(ty), "dk": _shared(dk, c["Hkv"]).to(ty), "dv": _shared(dv, c["Hkv"]).to(ty)}


def _values(x8, scale):
    """The values that 8-bit tokens stand for, in 32 bits."""
    B, H, M, d = x8.shape
    return (x8.float().view(B, H, M // BLOCK, BLOCK, d) * scale[..., None, None]).view(B, H, M, d)


def _plain_cached(s):
    c, H = s["case"], s["case"]["H"]
    (k8, ks), (v8, vs) = s["cache"]
    o, lse = _attend(s["q"].float(), _heads(_values(k8, ks), H), _heads(_values(v8, vs), H), s["lens"])[:2]
    return {"o": o.to(s["type"]), "lse": lse}


def _plain_append_one(x8, scale, x, pos):
    """The blocks that the new tokens touch, rounded anew; writes the cache, returns the new tokens' values."""
    B, H, n, d = x.shape
    cap = x8.shape[2]
    nb = (n + BLOCK - 2) // BLOCK + 1  # blocks that n tokens can touch
    first = (pos // BLOCK).long()
    at = (first[:, None] * BLOCK + torch.arange(nb * BLOCK, device=x.device)).clamp_(max=cap - 1)  # [B, nb * BLOCK]
    idx = at[:, None, :, None].expand(B, H, nb * BLOCK, d)
    blk = (first[:, None] + torch.arange(nb, device=x.device)).clamp_(max=cap // BLOCK - 1)[:, None].expand(B, H, nb)
    token = first[:, None] * BLOCK + torch.arange(nb * BLOCK, device=x.device)
    old = token < pos[:, None]
    new = (token >= pos[:, None]) & (token < pos[:, None] + n)
    src = (token - pos[:, None]).clamp_(0, n - 1)[:, None, :, None].expand(B, H, nb * BLOCK, d)
    fresh = torch.where(new[:, None, :, None], x.float().gather(2, src), 0.0).view(B, H, nb, BLOCK, d)
    held = old.view(B, 1, nb, BLOCK).any(3)
    was = scale.gather(2, blk)
    need = torch.exp2(torch.ceil(torch.log2(fresh.abs().amax((3, 4)) / 448.0)).clamp_(E_MIN, E_MAX))
    now = torch.where(held, torch.maximum(was, need), need)
    kept = x8.view(torch.uint8).gather(2, idx).view(torch.float8_e4m3fn).float().view(B, H, nb, BLOCK, d) * was[..., None, None]
    value = torch.where(old.view(B, 1, nb, BLOCK, 1), kept, fresh)
    held8 = (value / now[..., None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    write = old | new
    b, t = torch.nonzero(write, as_tuple=True)
    x8.view(torch.uint8)[b, :, token[b, t]] = held8.view(torch.uint8).view(B, H, nb * BLOCK, d)[b, :, t]
    b, t = torch.nonzero(write.view(B, nb, BLOCK).any(2), as_tuple=True)
    scale[b, :, first[b] + t] = now[b, :, t]
    back = (held8.float() * now[..., None, None]).view(B, H, nb * BLOCK, d)
    at = (pos.long() % BLOCK)[:, None] + torch.arange(n, device=x.device)
    return back.gather(2, at[:, None, :, None].expand(B, H, n, d))


def _plain_append(s):
    (k8, ks), (v8, vs) = s["cache"]
    k = _plain_append_one(k8, ks, s["k"], s["lens"])
    v = _plain_append_one(v8, vs, s["v"], s["lens"])
    return {"k": k.to(s["type"]), "v": v.to(s["type"]), "k_scale": ks, "v_scale": vs}


# --------------------------------------------------------------------- the package's operators


def _own(s):
    import block_sparse_attention_sa2_gb300 as sa2

    c = s["case"]
    if c["kind"] in ("cross", "train"):
        o, lse = sa2.cross_attn_fwd(s["q"], s["k"], s["v"], kv_len=s["kv_len"])
        if c["kind"] == "cross":
            return {"o": o, "lse": lse}
        dq, dk, dv = sa2.cross_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], kv_len=s["kv_len"])
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    (k8, ks), (v8, vs) = s["cache"]
    cache = sa2.KvCache8(k8, v8, ks, vs)
    if c["kind"] == "cached":
        o, lse = sa2.cache8_attn(s["q"], cache, s["kv_len"])
        return {"o": o, "lse": lse}
    sa2.cache8_append(cache, s["k"], s["v"], s["lens"])
    k, v = sa2.cache8_read(cache, s["lens"], c["n"], dtype=s["type"])
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}


def run(state):
    if own:
        return _own(state)
    return {"cross": _plain_cross, "train": _plain_cross, "cached": _plain_cached, "append": _plain_append}[state["case"]["kind"]](state)


def work(case):
    c, d = case, case["d"]
    lens = _lens(c)
    if c["kind"] == "append":
        new, kept = c["B"] * c["n"], sum(x % BLOCK for x in lens)
        # new tokens in and back out at 16 bits, their 8-bit form out and in again; the tokens of blocks that are extended, in and out
        return {"bytes": 2 * c["Hkv"] * d * (new * (2 + 1 + 1 + 2) + kept * 2), "flops": 0}
    size = 1 if c["kind"] == "cached" else 2
    rows, pairs = c["B"] * c["N"] * c["H"], c["N"] * c["H"] * sum(lens)
    q, kv = rows * d * 2, sum(lens) * c["Hkv"] * d * size
    if c["kind"] == "train":
        # q, dO in, O, dQ out; K, V in, dK, dV out
        return {"bytes": 4 * q + 4 * kv + rows * 4, "flops": 14 * pairs * d}
    return {"bytes": 2 * q + 2 * kv + rows * 4, "flops": 4 * pairs * d}


# ------------------------------------------------------- the definitions in 64 bits, head by head


def _exact_rows(q, k, v, scale):
    """softmax(scale q k^T) v of one head over keys that all count, with the LSE and the probabilities."""
    s = (q @ k.mT) * scale
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    return p @ v, lse, p


def _exact_held(v8, scale, e4m3_of=None):
    """One head's tokens from their 8-bit form."""
    return v8.double() * scale.double().repeat_interleave(BLOCK)[: v8.shape[0], None]


def _round_e4m3(x):
    """Nearest multiple of the e4m3 spacing at x, ties to even, by its definition."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    lens, dev = _lens(c), "cuda"
    if c["kind"] == "append":
        got = {}
        for name, (x8, scale) in zip("kv", s["cache"]):
            out = torch.empty((c["B"], c["Hkv"], c["n"], c["d"]), dtype=torch.float64, device=dev)
            for b in range(c["B"]):
                p, n = lens[b], c["n"]
                for j in range(p // BLOCK, (p + n - 1) // BLOCK + 1):
                    lo, hi = max(p, j * BLOCK), min(p + n, (j + 1) * BLOCK)
                    x = s[name][b, :, lo - p : hi - p].double()
                    amax = x.abs().amax((1, 2))
                    e = torch.floor(torch.log2(amax / 448)).clamp(E_MIN, E_MAX)
                    e = torch.where((amax > 448 * torch.exp2(e)) & (e < E_MAX), e + 1, e)
                    sc = torch.exp2(e)
                    if p > j * BLOCK:
                        sc = torch.maximum(sc, scale[b, :, j].double())
                    scale[b, :, j] = sc.float()
                    out[b, :, lo - p : hi - p] = _round_e4m3((x / sc[:, None, None]).clamp(-448, 448)) * sc[:, None, None]
            got[name] = out
            got[name + "_scale"] = scale.double()
        return got
    B, H, Hkv, N, d = c["B"], c["H"], c["Hkv"], c["N"], c["d"]
    pairs = H * N * sum(lens)
    if pairs * (14 if c["kind"] == "train" else 4) * d > 8e12:
        return None
    o = torch.zeros((B, H, N, d), dtype=torch.float64, device=dev)
    lse = torch.full((B, H, N), float("-inf"), dtype=torch.float64, device=dev)
    got = {"o": o, "lse": lse}
    if c["kind"] == "train":
        got["dq"] = torch.zeros_like(o)
        got["dk"], got["dv"] = (torch.zeros((B, Hkv, c["M"], d), dtype=torch.float64, device=dev) for _ in range(2))
    scale = d**-0.5
    for b in range(B):
        n = lens[b]
        if n == 0:
            continue
        for h in range(H):
            g = h * Hkv // H
            if c["kind"] == "cached":
                (k8, ks), (v8, vs) = s["cache"]
                k, v = _exact_held(k8[b, g, :n], ks[b, g]), _exact_held(v8[b, g, :n], vs[b, g])
            else:
                k, v = s["k"][b, g, :n].double(), s["v"][b, g, :n].double()
            q = s["q"][b, h].double()
            rows = max(1, int(4e8 // n))
            for r in range(0, N, rows):
                at = slice(r, r + rows)
                o[b, h, at], lse[b, h, at], p = _exact_rows(q[at], k, v, scale)
                if c["kind"] == "train":
                    do = s["do"][b, h, at].double()
                    dp = do @ v.mT
                    ds = p * (dp - (p * dp).sum(1, keepdim=True))
                    got["dq"][b, h, at] = ds @ k * scale
                    got["dk"][b, g, :n] += ds.mT @ q[at] * scale
                    got["dv"][b, g, :n] += p.mT @ do
    return got
