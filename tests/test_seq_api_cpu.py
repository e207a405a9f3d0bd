"""Host-side checks of the packed and paged entry points that need no GPU: refusals come
before any CUDA call, and accepted arguments reach the device check."""

import ctypes

import pytest
import torch

from exact_io_aware_74_b200 import fa2

P = 1 << 20  # a fake, aligned "device pointer": never dereferenced on these paths
E, U, W = fa2.FA2_ERR_INVALID_ARG, fa2.FA2_ERR_UNSUPPORTED, fa2.FA2_ERR_WORKSPACE
NO_DEVICE = (fa2.FA2_ERR_CUDA, fa2.FA2_ERR_ARCH)


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_74_b200 import build
    build.build()
    return fa2.load()


def rows(at, row=512, head=64):
    return fa2.FA2Packed(at * P, row, head)


def pages(at, block=8192, head=1024, row=64):
    return fa2.FA2Cache(at * P, block, head, row)


def needs_no_gpu():
    if torch.cuda.is_available():
        pytest.skip("these fake pointers are only safe without a device")


def fwd(lib, q=rows(1), k=rows(2), v=rows(3), o=rows(4), lse=5 * P, cu=6 * P, B=2, T=64, H=8, Hk=2, d=64,
        scale=0.1, causal=1, window=0, dtype=1):
    return lib.fa2_fwd_varlen(q, k, v, o, lse, cu, B, T, H, Hk, d, scale, causal, window, dtype, None)


BAD_SIZES = [(dict(B=0), E), (dict(T=-1), E), (dict(H=0), E), (dict(Hk=0), E), (dict(Hk=3), E),
             (dict(H=258, Hk=2), E), (dict(d=60), U), (dict(d=4), U), (dict(d=0), U), (dict(B=1 << 25), E),
             (dict(T=(1 << 30) + 1), E)]
BAD_MODES = [(dict(scale=0.0), E), (dict(scale=float("nan")), E), (dict(scale=float("inf")), E), (dict(causal=2), E),
             (dict(window=-1), E), (dict(window=4, causal=0), E), (dict(dtype=2), E)]


@pytest.mark.parametrize("kw,expect", BAD_SIZES + BAD_MODES + [
    (dict(d=264), U), (dict(lse=0), E), (dict(cu=0), E), (dict(cu=P + 2), E), (dict(q=rows(0)), E),
    (dict(k=fa2.FA2Packed(P + 8, 512, 64)), E), (dict(q=rows(1, row=500)), E), (dict(v=rows(3, row=32)), E),
    (dict(o=rows(4, head=68)), E), (dict(o=rows(1)), E), (dict(o=rows(2)), E), (dict(lse=3 * P), E),
    (dict(q=rows(1, row=1 << 38)), E), (dict(q=rows(1, row=-512)), E),
])
def test_forward_refusals(lib, kw, expect):
    assert fwd(lib, **kw) == expect


def test_forward_accepts(lib):
    assert fwd(lib, T=0, q=rows(0), k=rows(0)) == fa2.FA2_OK  # nothing to do
    needs_no_gpu()
    for kw in (dict(), dict(d=256, q=rows(1, 4096, 256), k=rows(2, 4096, 256), v=rows(3, 4096, 256),
                            o=rows(4, 4096, 256)), dict(window=5), dict(causal=0),
               dict(T=1, q=rows(1, row=3)),              # one row: its stride is not read
               dict(Hk=1, k=rows(2, head=0), v=rows(3, head=0)), dict(q=rows(1, row=64, head=64 * 64))):
        assert fwd(lib, **kw) in NO_DEVICE, kw


def bwd(lib, d=64, ws=32 * P, ws_bytes=None, B=2, T=64, H=8, Hk=2, scale=0.1, causal=1, window=0, dtype=1, **kw):
    names = ["q", "k", "v", "o", "do", "lse", "dq", "dk", "dv"]
    a = {n: rows(i + 1) for i, n in enumerate(names)}
    a["lse"] = 6 * P
    a.update(kw)
    if ws_bytes is None:
        ws_bytes = 1 << 30
    return lib.fa2_bwd_varlen(a["q"], a["k"], a["v"], a["o"], a["do"], a["lse"], a["dq"], a["dk"], a["dv"], 10 * P, ws,
                              ws_bytes, B, T, H, Hk, d, scale, causal, window, dtype, None)


@pytest.mark.parametrize("kw,expect", BAD_SIZES + BAD_MODES + [
    (dict(d=136), U), (dict(lse=0), E), (dict(do=rows(0)), E), (dict(dk=rows(8, row=12)), E),
    (dict(dq=rows(1)), E), (dict(dk=rows(7)), E), (dict(dv=rows(5)), E), (dict(ws=0), W), (dict(ws=P + 16), W),
    (dict(ws_bytes=8), W),
])
def test_backward_refusals(lib, kw, expect):
    assert bwd(lib, **kw) == expect


def test_backward_workspace(lib):
    size = fa2.fa2_bwd_varlen_workspace_size
    for T in (0, 1, 100, 5000):
        n = size(3, T, 8, 2, 64)
        assert n > 0 and n % 256 == 0
        assert bwd(lib, B=3, T=T, ws_bytes=n - 256) == (fa2.FA2_OK if T == 0 else W)
    assert size(3, 100, 8, 3, 64) == 0 and size(3, 100, 8, 2, 136) == 0 and size(0, 100, 8, 2, 64) == 0
    assert size(3, 1 << 20, 8, 2, 128) < (1 << 20) * 8 * (128 * 4 + 8) + (1 << 21)  # linear in T
    needs_no_gpu()
    assert bwd(lib, ws_bytes=size(2, 64, 8, 2, 64)) in NO_DEVICE


def paged(lib, q=rows(1), k=pages(2), v=pages(3), o=rows(4), lse=5 * P, cu=6 * P, lens=7 * P, table=8 * P, ws=9 * P,
          ws_bytes=1 << 30, B=2, T=64, H=8, Hk=2, d=64, blocks=10, block=16, most=4, scale=0.1, causal=1, window=0,
          dtype=1):
    return lib.fa2_fwd_paged(q, k, v, o, lse, cu, lens, table, ws, ws_bytes, B, T, H, Hk, d, blocks, block, most, scale,
                             causal, window, dtype, None)


@pytest.mark.parametrize("kw,expect", BAD_SIZES + BAD_MODES + [
    (dict(d=264), U), (dict(block=0), E), (dict(block=4), E), (dict(block=24), E), (dict(block=160), E),
    (dict(T=1 << 22, H=256, Hk=2, most=1 << 20), E),  # more than the kernel counts
    (dict(blocks=0), E), (dict(most=0), E), (dict(blocks=1 << 28, block=16), E), (dict(most=1 << 27), E),
    (dict(k=pages(0)), E), (dict(v=pages(3, row=8)), E), (dict(k=pages(2, head=1001)), E), (dict(lens=0), E),
    (dict(table=0), E), (dict(table=P + 1), E), (dict(o=rows(2)), E), (dict(o=rows(1)), E),
])
def test_paged_refusals(lib, kw, expect):
    assert paged(lib, **kw) == expect


def test_paged_accepts(lib):
    assert paged(lib, T=0) == fa2.FA2_OK
    size = fa2.fa2_fwd_paged_workspace_size
    assert size(2, 64, 8, 2, 64, 148) % 256 == 0 and size(2, 64, 8, 2, 64, 148) > 0
    assert size(2, 64, 8, 3, 64, 148) == 0 and size(2, 64, 8, 2, 264, 148) == 0
    needs_no_gpu()
    assert size(2, 64, 8, 2, 64, 0) == 0  # no device to ask
    for kw in (dict(), dict(block=128), dict(block=384), dict(window=9), dict(causal=0, most=1)):
        assert paged(lib, **kw) in NO_DEVICE, kw


def tables(lib, ctx=P, new=2 * P, free=3 * P, num_free=5, table=4 * P, cu=5 * P, lens=6 * P, pos=7 * P, slots=8 * P,
           used=9 * P, B=2, T=4, block=16, most=3):
    return lib.fa2_paged_tables(ctx, new, free, num_free, table, cu, lens, pos, slots, used, B, T, block, most, None)


@pytest.mark.parametrize("kw", [dict(ctx=0), dict(new=0), dict(free=0), dict(num_free=-1), dict(table=0), dict(cu=0),
                                dict(lens=0), dict(pos=0), dict(slots=0), dict(used=0), dict(B=0), dict(T=-1),
                                dict(block=0), dict(most=0), dict(slots=P + 2)])
def test_tables_refusals(lib, kw):
    assert tables(lib, **kw) == E


def append(lib, k=rows(1), v=rows(2), kc=pages(3), vc=pages(4), slots=5 * P, T=3, Hk=2, d=64, blocks=4, block=16):
    return lib.fa2_paged_append(k, v, kc, vc, slots, T, Hk, d, blocks, block, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), E), (dict(Hk=0), E), (dict(d=60), U), (dict(d=264), U), (dict(blocks=0), E), (dict(block=0), E),
    (dict(slots=0), E), (dict(k=rows(0)), E), (dict(kc=pages(1)), E), (dict(vc=pages(3)), E),
    (dict(kc=pages(3, row=20)), E), (dict(blocks=1 << 20, block=1 << 12), E),
])
def test_append_refusals(lib, kw, expect):
    assert append(lib, **kw) == expect


def test_tables_and_append_accept(lib):
    assert append(lib, T=0) == fa2.FA2_OK
    needs_no_gpu()
    assert append(lib) in NO_DEVICE and append(lib, block=7) in NO_DEVICE
    assert tables(lib) in NO_DEVICE and tables(lib, T=0, pos=0, slots=0) in NO_DEVICE
    assert tables(lib, free=0, num_free=0) in NO_DEVICE


def test_binding_refuses_other_tensors():
    """The checks of the Python binding, before the library is called."""
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        fa2.forward_varlen(q, q, q, cu, 0.1, True)
    with pytest.raises(ValueError):
        fa2.paged_append(q, q, q[None], q[None], cu)
    with pytest.raises(ValueError):
        fa2.paged_tables(cu, cu, cu, torch.zeros((2, 3), dtype=torch.int32), 4, 16)


def test_structs_are_laid_out_as_declared():
    assert ctypes.sizeof(fa2.FA2Packed) == 24 and ctypes.sizeof(fa2.FA2Cache) == 32
