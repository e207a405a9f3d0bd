"""NaN and infinities among the values that rows see, in the packed forward.

A row whose scores hold a NaN or a +inf has no finite softmax: the 64-bit reference is not
finite there, and neither may the result be, in O (NaN) and in LSE (NaN or +inf, never the -inf
of a row that sees no key).  Every other row stays within the bounds of packed_ref.py.
"""

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from packed_ref import assert_within, packed_forward
from test_varlen_gpu import make, ok

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf")]


def compare(o, lse, ro, rl, bo, bl):
    """Not finite where the reference is not, and within the bounds elsewhere."""
    rows = ~torch.isfinite(rl)  # [H, T]
    assert rows.any() and not rows.all()
    assert not torch.isfinite(ro).all(-1).t()[rows].any()
    assert torch.isnan(lse[rows]).logical_or(lse[rows] == float("inf")).all()
    assert torch.isnan(o.transpose(0, 1)[rows].float()).all()
    fine = ~rows
    assert_within(lse[fine], rl[fine], bl[fine], "LSE")
    assert_within(o.transpose(0, 1)[fine], ro.transpose(0, 1)[fine], bo.transpose(0, 1)[fine], "O")


# ------------------------------------------------------------------ packed

@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["query", "key"])
@pytest.mark.parametrize("lens,d", [([90, 200, 40], 64), ([90, 200, 40], 128), ([90, 200, 40], 256),
                                    ([1500, 90, 3000, 700, 2000], 64), ([1500, 90, 3000, 700, 2000], 128)],
                         ids=["one-tile-64", "one-tile-128", "one-tile-256", "two-tiles-64", "two-tiles-128"])
def test_packed(lens, d, where, bad):
    H, Hk = 8, 4
    q, k, v, _, cu = (t.clone() for t in make(lens, H, Hk, d, "bf16", 1))
    row = lens[0] + 60  # in the middle of the second sequence
    if where == "query":
        q[row, 5, 3] = bad
    else:
        q[..., 3] = q[..., 3].abs() + 0.5  # so that an infinite key gives every row that sees it +inf
        k[row, 2, 3] = bad
    o, lse = fa2.forward_varlen(q, k, v, cu, d ** -0.5, True)
    ok()
    compare(o, lse, *packed_forward(q, k, v, lens, d ** -0.5, True))
