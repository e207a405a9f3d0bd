"""NaN and +inf among the values that rows see, in the dense forward, window and decode calls.

A row whose scores hold a NaN or a +inf has no finite softmax: its O is NaN and its LSE NaN (or
+inf), however the keys are split; every other row is as the 64-bit reference has it (O max-abs
2e-2 in bf16, LSE 1e-3, the tolerances of the dense tests).
"""

import math

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from packed_ref import forward_one

pytestmark = pytest.mark.gpu

BAD = [float("nan"), float("inf")]


def inputs(B, H, Nq, Nk, d, where, bad):
    g = torch.Generator(device="cuda").manual_seed(Nq + Nk + d)
    q, k, v = (torch.randn((B, H, n, d), generator=g, device="cuda").to(torch.bfloat16) for n in (Nq, Nk, Nk))
    if where == "query":
        q[0, 1, Nq - 1, 3] = bad
    else:
        q[..., 3] = q[..., 3].abs() + 0.5  # so that an infinite key gives every row that sees it +inf
        k[0, 1, Nk - 2 if where == "late key" else 1, 3] = bad
    return q, k, v


def compare(q, k, v, o, lse, causal, window=0):
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)
    s, seen = 1 / math.sqrt(q.shape[3]), 0
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            ro, rl = forward_one(q[b, h].double(), k[b, h].double(), v[b, h].double(), s,
                                 k.shape[2] - q.shape[2], causal, window, q.dtype)[:2]
            bad = ~torch.isfinite(rl)
            seen += int(bad.sum())
            assert torch.isnan(o[b, h][bad].float()).all()
            assert (torch.isnan(lse[b, h][bad]) | (lse[b, h][bad] == float("inf"))).all()
            if not bad.all():
                assert float((o[b, h].double() - ro)[~bad].abs().max()) <= 2e-2
                assert float((lse[b, h].double() - rl)[~bad].abs().max()) <= 1e-3
    assert seen


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["query", "key", "late key"])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_forward(d, where, bad):
    q, k, v = inputs(2, 2, 300, 300, d, where, bad)
    for causal in (True, False):
        compare(q, k, v, *fa2.forward(q, k, v, 1 / math.sqrt(d), causal), causal)
    compare(q, k, v, *fa2.forward_window(q, k, v, 1 / math.sqrt(d), 50), True, 50)


@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("where", ["query", "key", "late key"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq,n_splits", [(1, 1), (1, 0), (20, 5), (40, 0), (100, 3), (300, 2)])
def test_decode(Nq, n_splits, d, where, bad):
    q, k, v = inputs(2, 2, Nq, 2500, d, where, bad)
    for causal in (True, False):
        compare(q, k, v, *fa2.forward_decode(q, k, v, 1 / math.sqrt(d), causal, n_splits), causal)


@pytest.mark.parametrize("where", ["query", "key"])
def test_8_bit_forward(where):
    """E4M3 has a NaN and no infinity."""
    x = [t.clamp(-2, 2) for t in inputs(1, 2, 300, 300, 64, where, 1.0)]
    q, k, v = (t.to(torch.float8_e4m3fn) for t in x)
    t, row = (q, 299) if where == "query" else (k, 1)
    t.view(torch.uint8)[0, 1, row, 3] = 0x7F
    for causal in (True, False):
        o, lse = fa2.forward_fp8(q, k, v, 0.125, causal, 1.0, 1.0, 1.0)
        assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)
        bad = torch.zeros((1, 2, 300), dtype=torch.bool, device="cuda")
        bad[0, 1, 299 if where == "query" else (slice(1, None) if causal else slice(None))] = True
        assert torch.isnan(o[bad].float()).all() and torch.isnan(lse[bad]).all()
        assert torch.isfinite(o[~bad].float()).all() and torch.isfinite(lse[~bad]).all()
