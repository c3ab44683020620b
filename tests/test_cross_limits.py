"""The limits that include/sa2.h states for cross attention are those that the calls have (no compute calls
here: each call that gets past the check in question is refused by a later one)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_cross_abi import ALIGN, FP16, INVALID, P, UNSUPPORTED, WORKSPACE, cache, fwd, lib, shape, tensor  # noqa: E402,F401


def test_key_heads_in_all(lib):  # noqa: F811
    """B and Hkv are limited one by one, in the backward as in the forward."""
    s = shape(B=32767, H=32767, Hkv=32767, N=1, M=1, d=64)
    t = tensor(heads=32767, tokens=1, d=64)
    size = lib.sa2_cross_bwd_workspace_size(s)
    assert size > 0
    assert lib.sa2_cross_attn_bwd(s, t, t, t, t, P, t, None, 0.0, t, t, t, P, 0, None) == WORKSPACE
    assert fwd(lib, s, q=t, o=t, k=t, v=t, ws=P + 8) == ALIGN


def test_strides_of_one_sequence(lib):  # noqa: F811
    s = shape(B=1, H=40, Hkv=40, N=1_700_000, M=1_700_000)
    t = tensor(heads=40, tokens=1_700_000, sn=40 * 128, sh=128)  # token-major
    assert fwd(lib, s, q=t, o=t, k=t, v=t, ws=P + 8) == ALIGN
    assert lib.sa2_cross_attn_bwd(s, t, t, t, t, P, t, None, 0.0, t, t, t, P, 0, None) == WORKSPACE
    one = shape(B=1, H=8, Hkv=8, N=(1 << 28) - 1, M=(1 << 28) - 1)
    t = tensor(heads=8, tokens=(1 << 28) - 1, sn=128)  # head-major, the largest stated length
    assert fwd(lib, one, q=t, o=t, k=t, v=t, ws=P + 8) == ALIGN


def test_strides_of_the_cache(lib):  # noqa: F811
    c = cache(sb=1 << 39, sh=128, sn=4 * 128)
    new = tensor(heads=4, tokens=7)
    assert lib.sa2_cache8_append(c, 7, 0, new, new, P + 2, None, None) == ALIGN


def test_strides_beyond_a_tensor_map(lib):  # noqa: F811
    """2^40 bytes; with shared key heads the stride of a key head's query heads is theirs together."""
    t = lambda **kw: tensor(**{**dict(heads=8, tokens=100, sn=128, sh=12800), **kw})  # noqa: E731
    most = (1 << 40) // 2
    call = lambda q: fwd(lib, q=q, o=q, ws=P + 8)  # noqa: E731
    assert call(t(sb=most - 8)) == ALIGN and call(t(sb=most)) == UNSUPPORTED
    assert call(t(sh=most // 2 - 8, sb=8)) == ALIGN and call(t(sh=most // 2, sb=8)) == UNSUPPORTED  # two to a key head
    kv = lambda **kw: tensor(**{**dict(heads=4, tokens=300, sn=128, sh=38400), **kw})  # noqa: E731
    assert fwd(lib, k=kv(sh=most - 8, sb=8), ws=P + 8) == ALIGN and fwd(lib, k=kv(sh=most, sb=8), ws=P + 8) == UNSUPPORTED
    assert fwd(lib, k=kv(sn=most, sh=8, sb=8), ws=P + 8) == UNSUPPORTED
    one = shape(B=1, H=4, Hkv=1)
    q = tensor(heads=4, tokens=100, sh=most - 8)
    assert fwd(lib, one, q=q, o=q, k=kv(), v=kv(), ws=P + 8) == ALIGN  # one key head: nothing is strided by the group
    assert fwd(lib, shape(dtype=FP16), q=t(sb=0), ws=P + 8) == INVALID
