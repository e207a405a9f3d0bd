"""NaN and infinities among the values that rows see, in the packed and paged forward.

A row whose scores hold a NaN or a +inf has no finite softmax: the 64-bit reference is not
finite there, and neither may the result be, in O (NaN) and in LSE (NaN or +inf, never the -inf
of a row that sees no key).  Every other row stays within the bounds of packed_ref.py.
"""

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from packed_ref import assert_within, packed_forward
from test_paged_gpu import Step, ok
from test_varlen_gpu import make

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


# ------------------------------------------------------------------ paged

def check_paged(context, new, H, Hk, d, where, bad, window=0, dtype="bf16"):
    """Request 1 holds the bad value: in its last query, or in a key that it sees."""
    s = Step(context, new, H, Hk, d, 16, dtype, seed=3)
    g = H // Hk
    row = sum(new[:2]) - 1
    if where == "query":
        s.q[row, g, 3] = bad
    else:
        s.q[..., 3] = s.q[..., 3].abs() + 0.5
        key = s.total[1] - 2 if where == "late key" else 1
        s.caches[1][0][key, 1, 3] = bad
        s.k_cache[int(s.table[1, key // 16]), 1, key % 16, 3] = bad
    for causal in (True, False):
        o, lse = s.run(causal, window if causal else 0)
        compare(o, lse, *packed_forward(s.q, None, None, s.new, s.scale, causal, window if causal else 0, s.caches))


# Short caches: every request's key tiles lie in one share.  Long ones: they are cut, into shares
# of two units where there are few requests, into longer ones where there are many.
SHORT, LONG, MANY = [60, 100, 5], [700, 4000, 90], [3000] * 40


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["query", "key", "late key"])
@pytest.mark.parametrize("context,new,d", [
    ([0, 3, 5], [20, 24, 22], 64), (LONG, [20, 24, 22], 128), (SHORT, [1, 1, 1], 256), (LONG, [1, 1, 1], 256),
    ([0, 3, 0], [50, 60, 70], 64), (LONG, [300, 200, 100], 64), (LONG, [300, 200, 100], 128)],
    ids=["one-tile", "one-tile-cut", "one-tile-256", "one-tile-256-cut", "two-tiles", "two-tiles-cut-64",
         "two-tiles-cut-128"])
def test_paged_tiles(context, new, d, where, bad):
    check_paged(context, new, 8, 2, d, where, bad)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["query", "key", "late key"])
@pytest.mark.parametrize("context", [SHORT, LONG, MANY], ids=["whole", "cut", "cut-seldom"])
@pytest.mark.parametrize("H,Hk,d,dtype", [(8, 2, 64, "bf16"), (8, 2, 128, "fp16"), (32, 2, 128, "bf16")])
def test_paged_few_rows(context, H, Hk, d, dtype, where, bad):
    check_paged(context, [1] * len(context), H, Hk, d, where, bad, dtype=dtype)
    if context is not SHORT and where != "key":
        check_paged(context, [1] * len(context), H, Hk, d, where, bad, window=300, dtype=dtype)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_queries_that_are_all_nan(d):
    """Every score of every row: no weight has a finite maximum to be measured from."""
    for context, new in ((SHORT, [1, 1, 1]), (LONG, [1, 1, 1]), (LONG, [30, 20, 22]), (LONG, [300, 200, 100])):
        s = Step(context, new, 8, 2, d, 16, "bf16", seed=4)
        s.q.fill_(float("nan"))
        o, lse = s.run()
        assert torch.isnan(o.float()).all() and torch.isnan(lse).all()
