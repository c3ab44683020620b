"""check_gradients of tests/cross_util.py lets a NaN element pass where it is told to leave the norm out (an
error that is NaN counts as none there); this one asks for finite gradients first."""
from tests.cross_util import check_gradients


def check_all_finite(got):
    for name, g in zip(("dq", "dk", "dv"), got):
        bad = ~g.isfinite()
        assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {g.numel()} elements not finite"


def check_finite_gradients(got, q, k, v, do, lens, scale=None, norm=True):
    check_all_finite(got)
    check_gradients(got, q, k, v, do, lens, scale, norm)
