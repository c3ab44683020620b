"""The limits that include/sa2.h states for cross attention are those that the calls have (no compute calls
here: each call that gets past the check in question is refused by a later one)."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_cross_abi import ALIGN, P, WORKSPACE, fwd, lib, shape, tensor  # noqa: E402,F401


def test_key_heads_in_all(lib):  # noqa: F811
    """B and Hkv are limited one by one, in the backward as in the forward."""
    s = shape(B=32767, H=32767, Hkv=32767, N=1, M=1, d=64)
    t = tensor(heads=32767, tokens=1, d=64)
    size = lib.sa2_cross_bwd_workspace_size(s)
    assert size > 0
    assert lib.sa2_cross_attn_bwd(s, t, t, t, t, P, t, None, 0.0, t, t, t, P, 0, None) == WORKSPACE
    assert fwd(lib, s, q=t, o=t, k=t, v=t, ws=P + 8) == ALIGN
