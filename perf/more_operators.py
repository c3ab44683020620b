"""Cases that measure attention within packed sequences, with its gradient, attention of new tokens over a
paged cache, and rotary positions.

``run`` computes each operator in plain torch operations (``own = False``) or through this package's entry
points (``own = True``) on the same inputs.  Sequences of different lengths lie one behind the other along the
token axis; ``seq`` ([B + 1] int32) says where each begins.  Four kinds of case:

* ``prompt``  O, LSE of whole sequences attending to themselves, causal, with shared key heads;
* ``train``   the same with dQ, dK, dV for a given dO: one training step of the layer;
* ``chunk``   new keys and values put into the pages of a cache, then O, LSE of the new tokens over all that
              the cache holds of their sequence up to each of them;
* ``rotary``  queries and keys turned by the angles of their positions (``grad``: and the gradients turned back).

A new token i of n, in a sequence of m tokens after the new ones, has position m - n + i.
"""
import math

import torch

own = False


def listed():
    return [
        # a few short prompts together, one of them empty: latency counts
        dict(name="prompt small", kind="prompt", B=4, T=256, H=8, Hkv=8, d=64, type="fp16", lens="ragged"),
        # a whole clip at 480p (21 x 30 x 52 tokens) frame by frame, key heads shared by four
        dict(name="prompt long", kind="prompt", B=1, T=32760, H=32, Hkv=8, d=128, type="bf16", lens="even"),
        # a batch of prompts packed without padding, odd lengths, three heads to a key head
        dict(name="prompt packed", kind="prompt", B=7, T=20011, H=24, Hkv=8, d=64, type="bf16", lens="ragged"),
        # a training step over one long sequence, a key head for each head
        dict(name="train long", kind="train", B=1, T=16380, H=12, Hkv=12, d=128, type="bf16", lens="even"),
        # a training step over a packed batch with shared key heads
        dict(name="train packed", kind="train", B=5, T=8190, H=32, Hkv=8, d=128, type="bf16", lens="ragged"),
        # many short captions, heads of 64
        dict(name="train short", kind="train", B=24, T=6001, H=16, Hkv=16, d=64, type="bf16", lens="ragged"),
        # one token for each sequence of a batch over long caches
        dict(name="chunk token", kind="chunk", B=16, T=16, M=32760, page=64, H=40, Hkv=8, d=128, type="bf16", lens="even", held="ragged"),
        # one token over one prompt: latency counts
        dict(name="chunk token small", kind="chunk", B=1, T=1, M=512, page=16, H=12, Hkv=12, d=128, type="bf16", lens="even", held="full"),
        # one frame's tokens (45 x 80) over a whole clip at 720p
        dict(name="chunk frame 720p", kind="chunk", B=1, T=3600, M=75600, page=128, H=40, Hkv=40, d=128, type="bf16", lens="even", held="full"),
        # a serving step: a piece of a prompt beside sequences that make single tokens
        dict(name="chunk mixed", kind="chunk", B=12, T=523, M=16001, page=32, H=32, Hkv=4, d=64, type="fp16", lens="one long", held="ragged"),
        # queries and keys of one layer of Wan2.1 14B at 720p: frame, row and column on channels of their own
        dict(name="rotary 720p", kind="rotary", B=1, N=75600, H=40, Hkv=40, d=128, rot=128, axes=3, layout="interleaved", scaling="none", type="bf16", grad=False),
        # a packed batch of text far behind the trained length, half of each head, both halves layout
        dict(name="rotary far", kind="rotary", B=3, N=1001, H=8, Hkv=2, d=128, rot=64, axes=1, layout="half", scaling="ramp", type="fp16", grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: every size over its logarithm, costs below the largest listed ones."""
    kind = rng.choice(("prompt", "prompt", "train", "train", "chunk", "chunk", "chunk", "rotary"))
    d = rng.choice((64, 128))
    hkv, group = rng.choice(((8, 4), (12, 1), (8, 3), (16, 1), (4, 8), (8, 5), (1, 7), (2, 16), (5, 1), (40, 1)))
    B = rng.choice((1, 1, 2, 3, 5, 8, 17, 32))
    ty = rng.choice(("bf16", "bf16", "fp16"))
    if kind == "rotary":
        axes = rng.choice((1, 1, 2, 3))
        layout = rng.choice(("interleaved", "half"))
        rot = rng.choice((d, d, d // 2, d // 2 + 16))
        return dict(kind=kind, B=rng.choice((1, 2, 3)), N=_log(rng, 1, 20000), H=hkv * group, Hkv=hkv, d=d, rot=rot, axes=axes, layout=layout,
                    scaling=rng.choice(("none", "linear", "base", "ramp")), type=rng.choice(("bf16", "fp16", "fp32")), grad=rng.random() < 0.5)
    while True:
        T = _log(rng, 1, 32760 if kind == "prompt" else 16380 if kind == "train" else 4000)
        c = dict(kind=kind, B=B, T=T, H=hkv * group, Hkv=hkv, d=d, type="bf16" if kind == "train" else ty,
                 lens=rng.choice(("even", "ragged", "one long")))
        if kind == "chunk":
            c.update(M=_log(rng, 64, 75600), page=rng.choice((16, 32, 64, 128, 256)), held=rng.choice(("full", "ragged")))
            if rng.random() < 0.4:
                c.update(T=B, lens="even")  # a single token for each
            if c["T"] > c["M"]:
                continue
        w = work(c)
        if w["flops"] <= (5.5e12 if kind != "train" else 2.9e12) and w["bytes"] <= 3.2e9:
            return c


def _lens(c):
    """Tokens of each sequence (chunk: new ones), T together."""
    T, B = c["T"], c["B"]
    if c["lens"] == "even":
        return [T * (b + 1) // B - T * b // B for b in range(B)]
    if c["lens"] == "one long":  # single tokens beside a long one, in the middle
        got = [1 if b < T - 1 else 0 for b in range(B)]
        got[B // 2] = 0
        got[B // 2] = T - sum(got)
        return got
    share = [0.05 + (0.61803 * (b + 1)) % 1 for b in range(B)]
    if B > 3:
        share[1] = 0.0  # a sequence without tokens
    at = [0]
    for x in share:
        at.append(at[-1] + x)
    cut = [int(T * x / at[-1]) for x in at]
    cut[-1] = T
    return [cut[b + 1] - cut[b] for b in range(B)]


def _held(c):
    """chunk: tokens that the cache holds of each sequence, the new ones among them."""
    M, new = c["M"], _lens(c)
    if c["held"] == "full":
        return [max(M, n) for n in new]
    got = [max(n, int(M * (1 - 0.61803 * b % 1))) for b, n in enumerate(new)]
    if len(got) > 2:
        got[2] = new[2]  # a sequence that begins with these tokens
    return got


def _type(c):
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["type"]]


def _sections(c):
    """Channels of each axis of a rotary case: even counts, the first gets what is left."""
    n = c["axes"]
    rest = c["rot"] // n // 2 * 2
    return [c["rot"] - rest * (n - 1)] + [rest] * (n - 1)


TRAINED = 4096  # rotary: positions of the trained context, and how many times that the scaled ones reach
FACTOR = 32.0
BASE = 10000.0


def _frequencies(c):
    """Angle of each channel pair for one step of its axis, the pair's axis, and the gain (64 bits)."""
    f, axis = [], []
    for a, n in enumerate(_sections(c)):
        base = BASE * FACTOR ** (n / (n - 2)) if c["scaling"] == "base" and n > 2 else BASE
        for i in range(n // 2):
            w = base ** (-2.0 * i / n)
            if c["scaling"] == "linear":
                w /= FACTOR
            elif c["scaling"] == "ramp":
                # pairs that turn at least 32 times over the trained context as they are, those that turn less than once slower
                r = TRAINED * w / (2 * math.pi)
                keep = min(max((r - 1.0) / (32.0 - 1.0), 0.0), 1.0)
                w = w * keep + w / FACTOR * (1 - keep)
            f.append(w)
            axis.append(a)
    return f, axis, 0.1 * math.log(FACTOR) + 1 if c["scaling"] == "ramp" else 1.0


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ty, d = _type(c), c["d"]

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(ty)

    s = dict(case=dict(c), type=ty)
    if c["kind"] == "rotary":
        # projections' outputs are token-major [B, N, H, d]: the operators take them as they lie
        s["q"], s["k"] = rnd(c["B"], c["N"], c["H"], d).transpose(1, 2), rnd(c["B"], c["N"], c["Hkv"], d).transpose(1, 2)
        if c["grad"]:
            s["dq"], s["dk"] = rnd(c["B"], c["N"], c["H"], d).transpose(1, 2), rnd(c["B"], c["N"], c["Hkv"], d).transpose(1, 2)
        reach = TRAINED if c["scaling"] == "none" else int(TRAINED * FACTOR)
        first = torch.randint(0, reach, (c["axes"], c["B"], 1), generator=g, device=dev)
        i = torch.arange(c["N"], device=dev)
        if c["axes"] == 1:
            s["pos"] = (first[0] + i).to(torch.int32)
        else:  # frame, row and column of tokens in raster order
            rows = (80, 45)[: c["axes"] - 1]
            at = []
            for n in rows:
                at.append(i % n)
                i = i // n
            s["pos"] = (torch.stack([i, *reversed(at)])[:, None] + first % 7).to(torch.int32)
        s["freq"] = _frequencies(c)
        if own:
            s["handle"] = _own_rotary(s)
        return s
    new = _lens(c)
    edges = [0]
    for n in new:
        edges.append(edges[-1] + n)
    s["seq"] = torch.tensor(edges, dtype=torch.int32, device=dev)
    s["q"], s["k"], s["v"] = (rnd(c["T"], h, d).transpose(0, 1) for h in (c["H"], c["Hkv"], c["Hkv"]))
    if c["kind"] == "train":
        s["do"] = rnd(c["T"], c["H"], d).transpose(0, 1)
    if c["kind"] == "chunk":
        held, page = _held(c), c["page"]
        per = [-(-n // page) for n in held]
        width = max(max(per), 1)
        # pages in the order in which a pool hands them out after a while: none in particular, some in nobody's use
        pages = sum(per) + 3
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.full((c["B"], width), -1, dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(per):
            table[b, :n] = order[at : at + n]
            at += n
        s["table"], s["kv_len"] = table, torch.tensor(held, dtype=torch.int32, device=dev)
        # a page's tokens lie head by head; what no sequence holds is of the same kind as what some do
        s["cache"] = tuple(torch.empty((pages, c["Hkv"], page, d), dtype=ty, device=dev).normal_(generator=g) for _ in range(2))
        s["max_new"] = max(new)
        if own:
            s["handle"] = _own_cache(s)
    return s


# ---------------------------------------------------------------- the operators in plain form


def _rows(H, keys):
    """Query rows at a time, so that the scores of all heads stay below 4 GB."""
    return max(1, int(2**30 // (H * max(keys, 1))))


def _attend(q, k, v, do=None):
    """n queries over m >= n keys, query i up to key m - n + i, [H, ., d] in 32 bits: O, LSE and, for dO, the gradients."""
    (H, n, d), (hkv, m, _) = q.shape, k.shape
    scale = 1.0 / math.sqrt(d)
    o, lse = torch.empty_like(q), torch.empty((H, n), device=q.device)
    kk, vv = (x.repeat_interleave(H // hkv, 0) if hkv != H else x for x in (k, v))
    if do is not None:
        dq, dk, dv = torch.empty_like(q), torch.zeros_like(kk), torch.zeros_like(vv)
    step = _rows(H, m)
    for r in range(0, n, step):
        e = min(r + step, n)
        keys = m - n + e
        s = torch.matmul(q[:, r:e], kk[:, :keys].transpose(1, 2)).mul_(scale)
        at = torch.arange(m - n + r, keys, device=q.device)
        s.masked_fill_(torch.arange(keys, device=q.device) > at[:, None], float("-inf"))
        mx = s.amax(2, keepdim=True)
        p = s.sub_(mx).exp_()
        l = p.sum(2, keepdim=True)
        p.div_(l)
        o[:, r:e] = torch.matmul(p, vv[:, :keys])
        lse[:, r:e] = (mx + torch.log(l)).squeeze(2)
        if do is not None:
            g = do[:, r:e]
            dv[:, :keys] += torch.matmul(p.transpose(1, 2), g)
            ds = torch.matmul(g, vv[:, :keys].transpose(1, 2))
            ds.sub_((g * o[:, r:e]).sum(2, keepdim=True)).mul_(p)
            dq[:, r:e] = torch.matmul(ds, kk[:, :keys]).mul_(scale)
            dk[:, :keys] += torch.matmul(ds.transpose(1, 2), q[:, r:e]).mul_(scale)
        del s, p
    if do is None:
        return o, lse
    dk, dv = (x.view(hkv, H // hkv, m, d).sum(1) for x in (dk, dv))
    return o, lse, dq, dk, dv


def _plain_packed(s):
    """Sequence by sequence; their places are known to the program that packed them."""
    c, ty = s["case"], s["type"]
    names = ["o", "lse"] + (["dq", "dk", "dv"] if c["kind"] == "train" else [])
    like = {"o": s["q"], "dq": s["q"], "dk": s["k"], "dv": s["k"]}
    out = {x: torch.empty_like(like[x]) if x in like else torch.empty((c["H"], c["T"]), device="cuda") for x in names}
    at = 0
    for n in _lens(c):
        if n == 0:
            continue
        w = slice(at, at + n)
        x = [s[t][:, w].float() for t in ("q", "k", "v") + (("do",) if c["kind"] == "train" else ())]
        for name, y in zip(names, _attend(*x)):
            out[name][:, w] = y.to(out[name].dtype)
        at += n
    return out


def _plain_chunk(s):
    c, page = s["case"], s["case"]["page"]
    o, lse = torch.empty_like(s["q"]), torch.empty((c["H"], c["T"]), device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(_lens(c), _held(c))):
        if n == 0:
            continue
        w = slice(at, at + n)
        t = torch.arange(m, device="cuda")
        pages, slot = s["table"][b, t // page].long(), t % page
        kv = []
        for name, x in zip("kv", s["cache"]):
            x[pages[m - n :], :, slot[m - n :]] = s[name][:, w].transpose(0, 1)
            kv.append(x[pages, :, slot].transpose(0, 1).float())
        y, l = _attend(s["q"][:, w].float(), *kv)
        o[:, w], lse[:, w] = y.to(s["type"]), l
        at += n
    return {"o": o, "lse": lse, "k_pages": s["cache"][0], "v_pages": s["cache"][1]}


def _turn(x, cos, sin, rot, half):
    """Pairs of the first rot channels by their angles; channels behind them as they are."""
    y = x.float().clone()
    if half:
        a, b = y[..., : rot // 2].clone(), y[..., rot // 2 : rot].clone()
        y[..., : rot // 2], y[..., rot // 2 : rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y.to(x.dtype)


def _plain_rotary(s):
    c = s["case"]
    f, axis, gain = s["freq"]
    # far positions: their angles in 64 bits
    f = torch.tensor(f, dtype=torch.float64, device="cuda")
    pos = s["pos"].double()
    pos = pos[None] if c["axes"] == 1 else pos
    angle = (pos[torch.tensor(axis, device="cuda")].permute(1, 2, 0) * f)[:, None]  # [B, 1, N, rot / 2]
    cos, sin = (torch.cos(angle) * gain).float(), (torch.sin(angle) * gain).float()
    half, rot = c["layout"] == "half", c["rot"]
    out = {"q": _turn(s["q"], cos, sin, rot, half), "k": _turn(s["k"], cos, sin, rot, half)}
    if c["grad"]:
        # channels that are not turned have no gain either
        out["dq"], out["dk"] = _turn(s["dq"], cos, -sin, rot, half), _turn(s["dk"], cos, -sin, rot, half)
    return out


# --------------------------------------------------------------------- the package's operators


def _own_rotary(s):
    import block_sparse_attention_sa2_gb300 as sa2

    c = s["case"]
    f, _, gain = s["freq"]
    sections = _sections(c)
    return sa2.Rotary(c["d"], f, axes=[n // 2 for n in sections], layout=c["layout"], gain=gain, device="cuda")


def _own_cache(s):
    import block_sparse_attention_sa2_gb300 as sa2

    return sa2.PagedCache(*s["cache"])


def _own(s):
    import block_sparse_attention_sa2_gb300 as sa2

    c = s["case"]
    if c["kind"] == "rotary":
        rotary = s.get("handle") or _own_rotary(s)
        q, k = sa2.rotary(rotary, s["pos"], s["q"], s["k"])
        out = {"q": q, "k": k}
        if c["grad"]:
            out["dq"], out["dk"] = sa2.rotary(rotary, s["pos"], s["dq"], s["dk"], inverse=True)
        return out
    if c["kind"] == "chunk":
        cache = s.get("handle") or _own_cache(s)
        sa2.paged_append(cache, s["k"], s["v"], s["seq"], s["kv_len"], s["table"])
        o, lse = sa2.paged_attn(s["q"], cache, s["seq"], s["kv_len"], s["table"], max_new=s["max_new"])
        return {"o": o, "lse": lse, "k_pages": s["cache"][0], "v_pages": s["cache"][1]}
    o, lse = sa2.packed_attn_fwd(s["q"], s["k"], s["v"], s["seq"])
    if c["kind"] == "prompt":
        return {"o": o, "lse": lse}
    dq, dk, dv = sa2.packed_attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], s["seq"])
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_packed, "train": _plain_packed, "chunk": _plain_chunk, "rotary": _plain_rotary}[state["case"]["kind"]](state)


def work(case):
    c, d = case, case["d"]
    size = 4 if c["type"] == "fp32" else 2
    if c["kind"] == "rotary":
        values = c["B"] * c["N"] * (c["H"] + c["Hkv"]) * d * (2 if c["grad"] else 1)
        return {"bytes": 2 * values * size + 4 * c["axes"] * c["B"] * c["N"], "flops": 0}
    new = _lens(c)
    q, kv = c["T"] * c["H"] * d * 2, c["T"] * c["Hkv"] * d * 2
    lse = c["T"] * c["H"] * 4
    if c["kind"] == "chunk":
        held = _held(c)
        pairs = c["H"] * sum(n * m - n * (n - 1) // 2 for n, m in zip(new, held))
        # new keys and values into the pages, and all that the attention reads of them
        read = sum(m for n, m in zip(new, held) if n) * c["Hkv"] * d * 2
        return {"bytes": 2 * q + lse + 2 * 2 * kv + 2 * read, "flops": 4 * pairs * d}
    pairs = c["H"] * sum(n * (n + 1) // 2 for n in new)
    if c["kind"] == "train":
        # q, dO in, O, dQ out; K, V in, dK, dV out
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 14 * pairs * d}
    return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * pairs * d}


# ------------------------------------------------------- the definitions in 64 bits, head by head


def _exact_turn(x, angle, gain, rot, layout):
    """Channel pairs as complex numbers times gain e^(i angle)."""
    y = x.double().clone()
    w = torch.polar(torch.full_like(angle, gain), angle)[:, None]
    part = y[..., :rot]
    if layout == "half":
        z = torch.complex(part[..., : rot // 2], part[..., rot // 2 :].contiguous()) * w
        y[..., :rot] = torch.cat((z.real, z.imag), -1)
    else:
        z = torch.view_as_complex(part.unflatten(-1, (rot // 2, 2)).contiguous()) * w
        y[..., :rot] = torch.view_as_real(z).flatten(-2)
    return y


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    dev = "cuda"
    if c["kind"] == "rotary":
        f, axis, gain = s["freq"]
        pos = s["pos"].double().reshape(c["axes"], c["B"], c["N"])
        angle = torch.stack([pos[a] * w for w, a in zip(f, axis)], -1)
        got = {x: _exact_turn(s[x], angle, gain, c["rot"], c["layout"]) for x in "qk"}
        if c["grad"]:
            got.update({x: _exact_turn(s[x], -angle, gain, c["rot"], c["layout"]) for x in ("dq", "dk")})
        return got
    H, Hkv, d, T = c["H"], c["Hkv"], c["d"], c["T"]
    train = c["kind"] == "train"
    if work(c)["flops"] > 9e12:
        return None
    z = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=dev)  # noqa: E731
    got = {"o": z(H, T, d), "lse": z(H, T)}
    if train:
        got.update(dq=z(H, T, d), dk=z(Hkv, T, d), dv=z(Hkv, T, d))
    if c["kind"] == "chunk":
        got.update(k_pages=None, v_pages=None)  # copies: not computed numbers
    seq = s["seq"].tolist()
    for b in range(c["B"]):
        lo, hi = seq[b], seq[b + 1]
        n = hi - lo
        if n == 0:
            continue
        for g in range(Hkv):
            k, v = s["k"][g, lo:hi].double(), s["v"][g, lo:hi].double()
            if c["kind"] == "chunk":
                before = int(s["kv_len"][b]) - n
                ids = s["table"][b, : -(-before // c["page"])].long()
                k, v = (torch.cat((x[ids, g].reshape(-1, d)[:before].double(), y)) for x, y in zip(s["cache"], (k, v)))
            m = k.shape[0]
            for h in range(g * H // Hkv, (g + 1) * H // Hkv):
                q = s["q"][h, lo:hi].double()
                step = max(1, min(2048, int(4e8 // m)))
                for r in range(0, n, step):
                    e = min(n, r + step)
                    to = m - n + e
                    x = (q[r:e] @ k[:to].mT) * d**-0.5
                    x += torch.full_like(x, float("-inf")).triu_(m - n + r + 1)
                    l = torch.logsumexp(x, 1)
                    p = torch.exp(x - l[:, None])
                    at = slice(lo + r, lo + e)
                    got["o"][h, at], got["lse"][h, at] = p @ v[:to], l
                    if train:
                        do = s["do"][h, at].double()
                        dp = do @ v[:to].mT
                        ds = p * (dp - (p * dp).sum(1, keepdim=True))
                        got["dq"][h, at] = ds @ k[:to] * d**-0.5
                        got["dk"][g, lo : lo + to] += ds.mT @ q[r:e] * d**-0.5
                        got["dv"][g, lo : lo + to] += p.mT @ do
    return got
