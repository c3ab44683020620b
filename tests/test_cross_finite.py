"""The gradients' check rejects elements that are not finite or were never written (CPU)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.cross_finite import check_finite_gradients  # noqa: E402
from tests.cross_util import gradients  # noqa: E402
from tests.test_cross_plain import case  # noqa: E402


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["all", "one", "behind the length"])
def test_what_is_not_finite_is_rejected(where, value, which):
    q, k, v, do = case()
    lens = [0, 8]
    got = [x.bfloat16() for x in gradients(q, k, v, do, lens)[0]]
    check_finite_gradients(got, q, k, v, do, lens, norm=False)
    at = {"all": (slice(None),), "one": (1, 1, 3, 5), "behind the length": (0 if which == 0 else 1, 0, -1)}[where]
    got[which][at] = value
    with pytest.raises(AssertionError, match="not finite"):
        check_finite_gradients(got, q, k, v, do, lens, norm=False)
