"""Packed sequences, the paged cache and rotary positions on the host: bad arguments are rejected before any launch,
workspace sizes cover their buffers, and the Python surface refuses what is not on a GPU (no compute calls here)."""
import ctypes
import struct

import pytest

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
P = 256  # a fake, aligned device pointer: never dereferenced on these paths
BF16, FP32, FP16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_sa2_gb300 import build_lib, sa2
    if not build_lib.up_to_date():
        build_lib.build()
    l = sa2.load_library()
    v, i, q, z, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    for name, args in (("sa2_packed_attn_fwd", [v, v, v, v, v, f, v, v, v, z, v]),
                       ("sa2_packed_attn_bwd", [v, v, v, v, v, v, v, v, f, v, v, v, v, z, v]),
                       ("sa2_paged_append", [v, i, i, v, v, v, v, v, v]),
                       ("sa2_paged_attn", [v, v, v, v, v, v, i, f, v, v, v, z, v]),
                       ("sa2_rotary_apply", [v, i, i, i, i, v, q, q, i, v, v, i, v, v, i, v])):
        getattr(l, name).argtypes, getattr(l, name).restype = args, ctypes.c_int
    for name, args in (("sa2_packed_fwd_workspace_size", [v]), ("sa2_packed_bwd_workspace_size", [v]),
                       ("sa2_paged_attn_workspace_size", [v, v, i, i])):
        getattr(l, name).argtypes, getattr(l, name).restype = args, z
    return l


def shape(B=3, H=8, Hkv=4, T=1000, d=128, dtype=BF16, causal=1, reserved=0):
    return struct.pack("8i", B, H, Hkv, T, d, dtype, causal, reserved)


def tensor(p=P, heads=8, tokens=1000, d=128, sh=None, sn=None, sb=0):
    sn = d if sn is None else sn
    return struct.pack("Pqqq", p, sb, tokens * sn if sh is None else sh, sn)


Q, KV = tensor(), tensor(heads=4)
MOST = 1 << 40


def fwd(lib, s=None, q=Q, k=KV, v=KV, seq=P, scale=0.0, o=Q, lse=P, ws=P, n=MOST):
    return lib.sa2_packed_attn_fwd(s or shape(), q, k, v, seq, scale, o, lse, ws, n, None)


def bwd(lib, s=None, q=Q, o=Q, lse=P, do=Q, seq=P, scale=0.0, dq=Q, dk=KV, ws=P, n=MOST):
    return lib.sa2_packed_attn_bwd(s or shape(), q, KV, KV, o, lse, do, seq, scale, dq, dk, KV, ws, n, None)


def test_packed_refusals(lib):
    for call in (fwd, bwd):
        for bad in (dict(B=0), dict(T=0), dict(H=9), dict(H=0), dict(Hkv=0), dict(reserved=1), dict(causal=2), dict(causal=-1)):
            assert call(lib, shape(**bad)) == INVALID, bad
        for bad in (dict(d=96), dict(dtype=FP32), dict(dtype=7), dict(H=260), dict(T=1 << 28), dict(B=1 << 20), dict(H=40000, Hkv=40000)):
            assert call(lib, shape(**bad)) == UNSUPPORTED, bad
        assert call(lib, q=None) == INVALID and call(lib, lse=None) == INVALID and call(lib, seq=None) == INVALID
        assert call(lib, scale=float("nan")) == INVALID and call(lib, scale=float("inf")) == INVALID
        assert call(lib, q=tensor(P + 8)) == ALIGN and call(lib, q=tensor(sn=132)) == ALIGN and call(lib, q=tensor(sn=64)) == INVALID
        assert call(lib, seq=P + 2) == ALIGN and call(lib, lse=P + 2) == ALIGN and call(lib, ws=P + 8) == ALIGN
        assert call(lib, q=tensor(sh=0)) == INVALID  # a broadcast head
    assert lib.sa2_packed_attn_fwd(None, Q, KV, KV, P, 0.0, Q, P, P, MOST, None) == INVALID
    assert bwd(lib, shape(dtype=FP16)) == UNSUPPORTED and bwd(lib, dk=tensor(p=0)) == INVALID and bwd(lib, do=None) == INVALID
    assert bwd(lib, o=tensor(p=P + 4)) == ALIGN
    # the stride of sequences is not used
    assert fwd(lib, q=tensor(sb=-3), ws=P + 8) == ALIGN


def test_workspaces(lib):
    size, bsize = lib.sa2_packed_fwd_workspace_size, lib.sa2_packed_bwd_workspace_size
    assert size(shape(d=80)) == 0 and size(None) == 0 and bsize(shape(dtype=FP16)) == 0 and bsize(None) == 0
    one = shape(B=1, H=2, Hkv=2, T=8000)  # few heads, long: split
    n = size(one)
    assert n >= 2 * 152 * 256 * (128 + 1) * 4 + 152 * 32
    t = tensor(heads=2, tokens=8000)
    assert fwd(lib, one, q=t, k=t, v=t, o=t, n=n - 4) == WORKSPACE and fwd(lib, one, q=t, k=t, v=t, o=t, ws=None) == WORKSPACE
    assert 0 < size(shape(B=2, H=40, Hkv=40, T=20000)) <= 4096  # a counter
    assert size(shape(B=1, H=2, Hkv=2, T=100)) == 0
    # statistics: B + T / tokens per tile records of 256 floats for each key head; behind them parts
    assert bsize(shape()) >= 4 * (3 + 1000 // 64) * 1024
    assert bwd(lib, n=bsize(shape()) - 4) == WORKSPACE and bwd(lib, ws=None) == WORKSPACE
    assert bsize(one) >= 2 * 2 * (8000 // 128 + 1) * 2 * 128 * 128 * 4


def pages(k=P, v=P, sp=None, sh=None, sn=None, pages=50, Hkv=4, page=64, d=128, dtype=BF16, reserved=0):
    sn = d if sn is None else sn
    sh = page * sn if sh is None else sh
    return struct.pack("PPqqqiiiiii", k, v, Hkv * sh if sp is None else sp, sh, sn, pages, Hkv, page, d, dtype, reserved)


def table(p=P, stride=16, width=16, reserved=0):
    return struct.pack("Pqii", p, stride, width, reserved)


def test_paged_refusals(lib):
    new = tensor(heads=4, tokens=7)
    app = lambda c=pages(), B=3, T=7, k=new, seq=P, kl=P, t=table(): lib.sa2_paged_append(c, B, T, k, new, seq, kl, t, None)  # noqa: E731

    def att(c=pages(), s=shape(), q=Q, seq=P, kl=P, t=table(), new=0, o=Q, lse=P, ws=P, n=MOST, scale=0.0):
        return lib.sa2_paged_attn(s, q, c, seq, kl, t, new, scale, o, lse, ws, n, None)

    for call in (app, att):
        for bad in (dict(k=0), dict(v=0), dict(pages=0), dict(Hkv=0), dict(page=0), dict(reserved=1), dict(sn=64), dict(sp=0)):
            assert call(c=pages(**bad)) == INVALID, bad
        for bad in (dict(d=96), dict(page=8), dict(page=48), dict(page=1 << 17), dict(dtype=FP32), dict(Hkv=40000)):
            assert call(c=pages(**bad)) == UNSUPPORTED, bad
        assert call(c=pages(k=P + 8)) == ALIGN and call(c=pages(v=P + 8)) == ALIGN and call(c=pages(sn=132)) == ALIGN
        for bad in (dict(p=0), dict(width=0), dict(reserved=1), dict(stride=-1)):
            assert call(t=table(**bad)) == INVALID, bad
        assert call(t=table(p=P + 2)) == ALIGN and call(t=table(width=1 << 22)) == UNSUPPORTED
        assert call(c=None) == INVALID and call(t=None) == INVALID and call(seq=None) == INVALID and call(kl=None) == INVALID
        assert call(kl=P + 1) == ALIGN and call(seq=P + 1) == ALIGN
    assert app(B=0) == INVALID and app(T=0) == INVALID and app(k=None) == INVALID and app(k=tensor(P + 2, 4, 7)) == ALIGN
    assert app(T=1 << 28) == UNSUPPORTED and app(B=1 << 20) == UNSUPPORTED
    assert att(s=shape(d=64)) == INVALID and att(s=shape(dtype=FP16)) == INVALID and att(s=shape(Hkv=2)) == INVALID
    assert att(new=-1) == INVALID and att(lse=None) == INVALID and att(q=None) == INVALID and att(scale=float("nan")) == INVALID
    assert att(ws=P + 8) == ALIGN
    size = lib.sa2_paged_attn_workspace_size
    # single tokens over long caches: parts of 16 rows; tiles of 256 for more
    few, more = size(shape(T=3), pages(pages=3000), 1000, 1), size(shape(T=300), pages(pages=3000), 1000, 100)
    assert 2 * 152 * 16 * 129 * 4 <= few < 2 * 152 * 256 * 129 * 4 <= more
    assert size(shape(T=3), pages(), 16, 1) == 0 and size(None, pages(), 16, 1) == 0 and size(shape(), None, 16, 1) == 0
    one = tensor(tokens=3)
    assert att(s=shape(T=3), c=pages(pages=3000), t=table(width=1000, stride=1000), new=1, q=one, o=one, n=few - 4) == WORKSPACE


def rotary(p=P, n=32, axes=1, layout=0, gain=1.0):
    return struct.pack("Piiif", p, n, axes, layout, gain)


def test_rotary_refusals(lib):
    x = tensor(tokens=10, sb=8 * 10 * 128)

    def call(r=rotary(), dtype=BF16, B=2, N=10, d=128, pos=P, pa=20, pb=10, H=8, x=x, y=x, H2=0, x2=None, y2=None, inv=0):
        return lib.sa2_rotary_apply(r, dtype, B, N, d, pos, pa, pb, H, x, y, H2, x2, y2, inv, None)

    for bad in (dict(p=0), dict(n=0), dict(axes=0), dict(layout=2), dict(gain=float("inf"))):
        assert call(r=rotary(**bad)) == INVALID, bad
    for bad in (dict(B=0), dict(N=0), dict(H=0), dict(H2=-1), dict(pos=None), dict(pa=-1), dict(pb=-1), dict(inv=2), dict(x=None), dict(y=None),
                dict(r=None), dict(H2=3)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(dtype=7), dict(d=100), dict(d=1032), dict(r=rotary(n=65)), dict(r=rotary(n=12, layout=1)), dict(B=1 << 20, N=1 << 10)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(x=tensor(P + 2, tokens=10, sb=8 * 10 * 128)) == ALIGN and call(r=rotary(p=P + 8)) == ALIGN and call(pos=P + 2) == ALIGN
    assert call(y=tensor(tokens=10, sb=8 * 10 * 128, sh=128, sn=1024)) == INVALID  # the same memory under other strides


def test_python_refuses_tensors_that_are_not_on_a_gpu(lib):
    import block_sparse_attention_sa2_gb300 as sa2
    q = torch.zeros((2, 3, 64), dtype=torch.bfloat16)
    seq, one = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    c = sa2.PagedCache.empty(4, 2, 16, 64, "cpu")
    assert c.shape == (4, 2, 16, 64) and c.k.dtype == torch.bfloat16
    tab = torch.zeros((1, 2), dtype=torch.int32)
    r = sa2.Rotary(64, [1.0], device="cpu")
    for f in (lambda: sa2.packed_attn_fwd(q, q, q, seq), lambda: sa2.packed_attn_bwd(q, q, q, q, q, q, seq),
              lambda: sa2.paged_append(c, q, q, seq, one, tab), lambda: sa2.paged_attn(q, c, seq, one, tab),
              lambda: sa2.rotary(r, one, q), lambda: sa2.packed_attn_fwd(q.float(), q, q, seq),
              lambda: sa2.packed_attn_fwd(q[None], q, q, seq), lambda: sa2.packed_attn_fwd(None, q, q, seq),
              lambda: sa2.packed_attn_fwd(q, q, q, seq[:1]), lambda: sa2.packed_attn_fwd(q, q, q, None),
              lambda: sa2.PagedCache(c.k, c.v[:, :, :8]), lambda: sa2.PagedCache(c.k.transpose(2, 3), c.v.transpose(2, 3)),
              lambda: sa2.PagedCache(c.k[0], c.v[0]), lambda: sa2.PagedCache(c.k.float(), c.v.float())):
        with pytest.raises(ValueError):
            f()
