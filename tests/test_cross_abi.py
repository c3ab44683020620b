"""Cross and cache attention on the host: bad arguments are rejected before any launch, workspace sizes
cover their buffers, and the Python surface refuses what is not on a GPU (no compute calls here)."""
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
    v, i, z, f = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
    for name, args in (("sa2_cross_attn_fwd", [v, v, v, v, v, f, v, v, v, z, v]),
                       ("sa2_cross_attn_bwd", [v, v, v, v, v, v, v, v, f, v, v, v, v, z, v]),
                       ("sa2_cache8_append", [v, i, i, v, v, v, v, v]), ("sa2_cache8_read", [v, i, i, v, v, v, v]),
                       ("sa2_cache8_attn", [v, v, v, v, f, v, v, v, z, v])):
        getattr(l, name).argtypes, getattr(l, name).restype = args, ctypes.c_int
    for name in ("sa2_cross_fwd_workspace_size", "sa2_cross_bwd_workspace_size"):
        getattr(l, name).argtypes, getattr(l, name).restype = [v], z
    return l


def shape(B=2, H=8, Hkv=4, N=100, M=300, d=128, dtype=BF16, reserved=0):
    return struct.pack("8i", B, H, Hkv, N, M, d, dtype, reserved)


def tensor(p=P, heads=8, tokens=100, d=128, sb=None, sh=None, sn=None):
    sn = d if sn is None else sn
    sh = tokens * sn if sh is None else sh
    return struct.pack("Pqqq", p, heads * sh if sb is None else sb, sh, sn)


Q, KV = tensor(), tensor(heads=4, tokens=300)


def fwd(lib, s=None, q=Q, k=KV, v=KV, kv_len=None, scale=0.0, o=Q, lse=P, ws=P, n=1 << 40):
    return lib.sa2_cross_attn_fwd(s or shape(), q, k, v, kv_len, scale, o, lse, ws, n, None)


def bwd(lib, s=None, q=Q, do=Q, dk=KV, lse=P, ws=P, n=1 << 40, scale=0.0):
    return lib.sa2_cross_attn_bwd(s or shape(), q, KV, KV, Q, lse, do, None, scale, Q, dk, KV, ws, n, None)


def test_forward_refusals(lib):
    for bad in (dict(B=0), dict(N=0), dict(M=0), dict(H=9), dict(H=0), dict(Hkv=0), dict(reserved=1)):
        assert fwd(lib, shape(**bad)) == INVALID, bad
    for bad in (dict(d=96), dict(dtype=FP32), dict(dtype=7), dict(H=260, Hkv=4), dict(N=1 << 28), dict(M=1 << 28),
                dict(B=40000)):
        assert fwd(lib, shape(**bad)) == UNSUPPORTED, bad
    assert fwd(lib, q=None) == INVALID and fwd(lib, lse=None) == INVALID and fwd(lib, o=tensor(p=0)) == INVALID
    assert fwd(lib, scale=float("nan")) == INVALID and fwd(lib, scale=float("inf")) == INVALID
    assert fwd(lib, k=tensor(P + 8, 4, 300)) == ALIGN and fwd(lib, q=tensor(sn=132)) == ALIGN
    assert fwd(lib, kv_len=P + 2) == ALIGN and fwd(lib, lse=P + 2) == ALIGN and fwd(lib, ws=P + 8) == ALIGN
    assert fwd(lib, q=tensor(sn=64)) == INVALID  # rows overlap
    assert fwd(lib, k=tensor(heads=4, tokens=300, sb=0)) == INVALID  # a broadcast batch
    assert fwd(lib, k=tensor(heads=4, tokens=300, sh=-128)) == INVALID
    # strides of dimensions of size 1 are ignored: refused only for the workspace
    one = shape(B=1, H=1, Hkv=1, N=1, M=4000)
    t = tensor(heads=1, tokens=1, sb=-5, sh=3, sn=7)
    assert fwd(lib, one, q=t, o=t, k=tensor(heads=1, tokens=4000, sb=1, sh=9), v=tensor(heads=1, tokens=4000), n=0) == WORKSPACE
    assert fwd(lib, one, q=t, o=t, k=tensor(heads=1, tokens=4000), v=tensor(heads=1, tokens=4000), ws=None) == WORKSPACE


def test_workspaces(lib):
    size = lib.sa2_cross_fwd_workspace_size
    assert size(shape()) == 0 and size(shape(d=80)) == 0 and size(None) == 0
    split = size(shape(B=1, H=8, Hkv=8, N=64, M=32760))
    assert split >= (152 + 8) * 256 * (128 + 1) * 4
    assert fwd(lib, shape(B=1, H=8, Hkv=8, N=64, M=32760), q=tensor(tokens=64), o=tensor(tokens=64),
               k=tensor(heads=8, tokens=32760), v=tensor(heads=8, tokens=32760), n=split - 4) == WORKSPACE
    few = size(shape(B=1, H=8, Hkv=8, N=1, M=32760))
    assert 0 < few < split  # slots of 16 rows instead of 256
    bsize = lib.sa2_cross_bwd_workspace_size
    assert bsize(shape(dtype=FP16)) == 0
    tiles = 2 * 4 * 2  # B * Hkv * ceil(100 / 64): two heads share a key head, 64 tokens a tile
    assert bsize(shape()) >= tiles * 256 * 4
    assert bwd(lib, n=bsize(shape()) - 4) == WORKSPACE and bwd(lib, ws=None) == WORKSPACE


def test_backward_refusals(lib):
    assert bwd(lib, shape(dtype=FP16)) == UNSUPPORTED and bwd(lib, shape(dtype=FP32)) == UNSUPPORTED
    assert bwd(lib, shape(d=32)) == UNSUPPORTED and bwd(lib, shape(H=7)) == INVALID
    assert bwd(lib, do=None) == INVALID and bwd(lib, lse=None) == INVALID and bwd(lib, dk=tensor(p=0)) == INVALID
    assert bwd(lib, scale=float("nan")) == INVALID
    assert bwd(lib, do=tensor(p=P + 4)) == ALIGN and bwd(lib, lse=P + 1) == ALIGN


def cache(k=P, v=P, ks=P, vs=P, sb=4 * 300 * 128, sh=300 * 128, sn=128, B=2, Hkv=4, C=300, d=128):
    return struct.pack("PPPPqqqiiii", k, v, ks, vs, sb, sh, sn, B, Hkv, C, d)


def test_cache_refusals(lib):
    new = tensor(heads=4, tokens=7)
    app = lambda c=cache(), n=7, dt=BF16, k=new, v=new, pos=P, cnt=None: lib.sa2_cache8_append(c, n, dt, k, v, pos, cnt, None)  # noqa: E731
    read = lambda c=cache(), n=7, dt=BF16, k=new, pos=P: lib.sa2_cache8_read(c, n, dt, k, new, pos, None)  # noqa: E731
    att = lambda c=cache(), s=shape(), q=Q, kl=P: lib.sa2_cache8_attn(s, q, c, kl, 0.0, Q, P, P, 1 << 40, None)  # noqa: E731
    for call in (app, read, att):
        assert call(c=cache(k=0)) == INVALID and call(c=cache(vs=0)) == INVALID and call(c=cache(C=0)) == INVALID
        assert call(c=cache(d=32)) == UNSUPPORTED and call(c=cache(B=40000)) == UNSUPPORTED
        assert call(c=cache(k=P + 8)) == ALIGN and call(c=cache(sn=136)) == ALIGN and call(c=cache(ks=P + 2)) == ALIGN
        assert call(c=cache(sn=64)) == INVALID and call(c=None) == INVALID
    for call in (app, read):
        assert call(n=0) == INVALID and call(pos=None) == INVALID and call(dt=FP32) == UNSUPPORTED
        assert call(k=None) == INVALID and call(k=tensor(P + 2, 4, 7)) == ALIGN and call(pos=P + 2) == ALIGN
    assert app(cnt=P + 1) == ALIGN
    assert att(kl=None) == INVALID and att(s=shape(M=301)) == INVALID and att(s=shape(B=1)) == INVALID
    assert att(s=shape(d=64)) == INVALID and att(q=None) == INVALID


def test_self_attention_calls_still_refuse_fp16(lib):
    from block_sparse_attention_sa2_gb300 import sa2
    s = sa2.Shape(1, 2, 1000, 128, 128, 64, FP16, 0, 2 * 1000 * 128, 1000 * 128, 128)
    assert lib.sa2_fwd_workspace_size(ctypes.byref(s)) == 0
    with pytest.raises(ValueError):
        sa2.make_shape(torch.zeros(1, 1, 4, 64, dtype=torch.float16), 128, 64)


def test_python_refuses_tensors_that_are_not_on_a_gpu(lib):
    import block_sparse_attention_sa2_gb300 as sa2
    q = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    c = sa2.KvCache8.empty(1, 2, 70, 64, "cpu")
    assert c.shape == (1, 2, 70, 64) and c.k_scale.shape == (1, 2, 2) and c.k.dtype == torch.float8_e4m3fn
    for f in (lambda: sa2.cross_attn_fwd(q, q, q), lambda: sa2.cross_attn_bwd(q, q, q, q, q, q),
              lambda: sa2.cache8_append(c, q, q, i), lambda: sa2.cache8_read(c, i, 3), lambda: sa2.cache8_attn(q, c, i),
              lambda: sa2.cross_attn_fwd(q.float(), q, q), lambda: sa2.cross_attn_fwd(q[0], q, q),
              lambda: sa2.cross_attn_fwd(None, q, q), lambda: sa2.cache8_read(c, i, -1),
              lambda: sa2.cache8_read(c, i, 3, dtype=torch.float32),
              lambda: sa2.KvCache8(c.k, c.v[:, :, :64], c.k_scale, c.v_scale),
              lambda: sa2.KvCache8(c.k.transpose(2, 3), c.v.transpose(2, 3), c.k_scale, c.v_scale),
              lambda: sa2.KvCache8(c.k, c.v, c.k_scale[:, :, :1], c.v_scale),
              lambda: sa2.KvCache8(c.k, c.v, c.k_scale, c.v_scale.double()),
              lambda: sa2.KvCache8(c.k[0], c.v[0], c.k_scale, c.v_scale)):
        with pytest.raises(ValueError):
            f()
