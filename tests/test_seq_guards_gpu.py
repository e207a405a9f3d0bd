"""Packed calls with bad offsets write nothing outside their outputs and workspace."""

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from test_varlen_gpu import make, ok

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


@pytest.mark.parametrize("T,H,Hk", [(300, 4, 2), (20000, 4, 4)], ids=["cut-tiles", "whole-tiles"])
@pytest.mark.parametrize("d", [64, 128])
def test_bad_offsets_of_the_packed_calls(T, H, Hk, d):
    """Offsets that fall, repeat or leave the tensors (the results are unspecified): rows before
    and behind every output and bytes around the workspace keep what they held."""
    q, k, v, do, _ = make([T], H, Hk, d, "bf16", 15)
    outer = {n: torch.full((T + 2, h, d), 7.0, dtype=torch.bfloat16, device="cuda")
             for n, h in (("o", H), ("dq", H), ("dk", Hk), ("dv", Hk))}
    o, dq, dk, dv = (outer[n][1:T + 1] for n in ("o", "dq", "dk", "dv"))
    lse_buf = torch.full((H * T + 2,), 7.0, device="cuda")
    lse = lse_buf[1:-1].view(H, T)
    need = fa2.fa2_bwd_varlen_workspace_size(3, T, H, Hk, d)
    ws_buf = torch.full((need + 512,), 199, dtype=torch.uint8, device="cuda")
    ws = ws_buf[256:256 + need]
    for at in ([0, T, 0, T], [-5, T // 3, TOP, 40], [T - 10, 20, T, -TOP - 1], [0, T, T, T], [TOP, TOP, 0, T],
               [T, 0, T, 0]):
        cu = torch.tensor(at, dtype=torch.int32, device="cuda")
        for causal, window in ((True, 0), (False, 0), (True, 70)):
            o.zero_()  # rows that a call leaves out: finite
            lse.zero_()
            assert fa2.fa2_fwd_varlen(q, k, v, o, lse, cu, 0.1, causal, window) == fa2.FA2_OK
            ok()
            assert fa2.fa2_bwd_varlen(q, k, v, o, do, lse, dq, dk, dv, cu, ws, 0.1, causal, window) == fa2.FA2_OK
            ok()
            for n, x in outer.items():
                assert (x[0] == 7).all() and (x[-1] == 7).all(), n
            assert lse_buf[0] == 7 and lse_buf[-1] == 7
            assert (ws_buf[:256] == 199).all() and (ws_buf[256 + need:] == 199).all()
