"""Raw handles of the default stream: outputs and workspaces of a call belong to it."""

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from test_paged_gpu import Step
from test_varlen_gpu import make, ok

pytestmark = pytest.mark.gpu

# 0, and 1, which is the same stream under its name of cudaStreamLegacy
HANDLES = [0, 1]


@pytest.mark.parametrize("handle", HANDLES)
def test_memory_is_allocated_on_the_default_stream(handle):
    t = torch.zeros(1, device="cuda")
    assert torch.cuda.default_stream().cuda_stream == 0
    with torch.cuda.stream(torch.cuda.Stream()):
        with fa2._home(t, handle):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        with fa2._home(t, torch.cuda.default_stream()):
            assert torch.cuda.current_stream() == torch.cuda.default_stream()


@pytest.mark.parametrize("handle", HANDLES)
def test_calls_on_the_default_stream_while_another_is_current(handle):
    """The current stream allocates and fills tensors of the outputs' and workspaces' sizes."""
    q, k, v, do, cu = make([300, 90, 1, 700], 4, 2, 64, "bf16", 16)
    s = Step([3000, 700, 0, 90], [1, 40, 130, 1], 8, 2, 128, 16, "bf16", seed=30)
    paged = s.run()
    o, lse = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    g = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.1, True)
    torch.cuda.synchronize()
    sizes = (fa2.fa2_bwd_varlen_workspace_size(4, q.shape[0], 4, 2, 64),
             fa2.fa2_fwd_paged_workspace_size(4, s.q.shape[0], 8, 2, 128))
    outs = []
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(40):
            a = fa2.forward_varlen(q, k, v, cu, 0.1, True, stream=handle)
            b = fa2.backward_varlen(q, k, v, *a[:1], do, a[1], cu, 0.1, True, stream=handle)
            c = fa2.forward_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.lens, s.scale, True, stream=handle)
            outs.append(a + b[1:] + c)
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in sizes:
                    torch.full((n,), 255, dtype=torch.uint8, device="cuda")
                torch.full_like(do, 3)
    torch.cuda.synchronize()
    ok()
    for got in outs:
        assert all(torch.equal(x, y) for x, y in zip(got, (o, lse) + g[1:] + paged))
