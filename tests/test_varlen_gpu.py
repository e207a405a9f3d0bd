"""Packed-sequence attention (fa2_fwd_varlen, fa2_bwd_varlen) against the 64-bit reference.

Bounds: see packed_ref.py.
"""

import math
import random

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from packed_ref import assert_within, packed_backward, packed_forward

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def make(lens, H, Hk, d, dtype, seed, extra=0):
    """Slices of one projection, as a model holds them, and the offsets."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + extra
    qkv = torch.randn((T, H + 2 * Hk, d), generator=g, device="cuda").to(DT[dtype])
    do = torch.randn((T, H, d), generator=g, device="cuda").to(DT[dtype])
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], do, torch.tensor(cu, dtype=torch.int32, device="cuda")


def ok():
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)


def check_forward(lens, H, Hk, d, dtype, causal, window, seed):
    q, k, v, _, cu = make(lens, H, Hk, d, dtype, seed)
    s = 1 / math.sqrt(d)
    o, lse = fa2.forward_varlen(q, k, v, cu, s, causal, window)
    ok()
    ro, rl, bo, bl = packed_forward(q, k, v, lens, s, causal, window)
    assert_within(lse, rl, bl, "LSE")
    assert_within(o, ro, bo, "O")


def check_backward(lens, H, Hk, d, dtype, causal, window, seed):
    q, k, v, do, cu = make(lens, H, Hk, d, dtype, seed)
    s = 1 / math.sqrt(d)
    o, lse = fa2.forward_varlen(q, k, v, cu, s, causal, window)
    got = fa2.backward_varlen(q, k, v, o, do, lse, cu, s, causal, window)
    ok()
    ref, bound = packed_backward(q, k, v, do, lens, s, causal, window)
    for name, x, r, b in zip(("dQ", "dK", "dV"), got, ref, bound):
        assert_within(x, r, b, name)


LENS = [[1], [0, 1, 2], [127, 128, 129], [5, 0, 300, 64, 1], [700, 260], [0, 0, 33, 0], [1] * 40,
        [513, 3, 1000]]
MODES = [(True, 0), (False, 0), (True, 1), (True, 100)]


@pytest.mark.parametrize("causal,window", MODES)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:5])))
@pytest.mark.parametrize("d", [64, 128])
def test_forward(lens, d, causal, window):
    check_forward(lens, 4, 2, d, "bf16", causal, window, seed=sum(lens) + d)


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (6, 2), (8, 8), (7, 1), (20, 4), (128, 1), (65, 1)])
@pytest.mark.parametrize("lens", [[3, 200, 131], [1, 1, 2]], ids=lambda x: "-".join(map(str, x)))
def test_forward_head_groups(lens, H, Hk):
    check_forward(lens, H, Hk, 64, "bf16", True, 0, seed=H)
    check_forward(lens, H, Hk, 128, "fp16", True, 50, seed=H + 1)


@pytest.mark.parametrize("d", [8, 24, 40, 72, 96, 120, 136, 192, 200, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_forward_head_dims(d, dtype):
    check_forward([150, 0, 290, 1], 6, 2, d, dtype, True, 0, seed=d)
    check_forward([150, 290], 2, 2, d, dtype, False, 0, seed=d + 1)


@pytest.mark.parametrize("causal,window", MODES)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[:5])))
@pytest.mark.parametrize("d", [64, 128])
def test_backward(lens, d, causal, window):
    check_backward(lens, 4, 2, d, "bf16", causal, window, seed=sum(lens) + d)


@pytest.mark.parametrize("H,Hk", [(1, 1), (4, 1), (6, 2), (8, 8), (7, 1), (128, 1)])
@pytest.mark.parametrize("d,dtype", [(64, "fp16"), (128, "bf16"), (96, "fp16"), (40, "bf16"), (8, "bf16")])
def test_backward_head_groups_and_dims(H, Hk, d, dtype):
    check_backward([3, 200, 131, 0, 1], H, Hk, d, dtype, True, 0, seed=H + d)
    check_backward([140, 20], H, Hk, d, dtype, False, 0, seed=H + d + 1)


@pytest.mark.parametrize("B", [96, 97, 256, 257, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_many_sequences(B, d):
    """More sequences than a scheduling warp keeps the counts of, empty ones among them."""
    r = random.Random(B)
    lens = [r.choice([0, 0, 1, 2, 7, 40]) for _ in range(B)]
    lens[B // 2] = 700
    lens[-1] = r.choice([0, 150])
    check_forward(lens, 2, 1, d, "bf16", True, 0, seed=B)
    check_backward(lens, 2, 1, d, "bf16", True, 0, seed=B + 1)
    few = [0] * B
    few[B // 3], few[-2] = 2, 1  # far more sequences than rows
    check_forward(few, 2, 2, d, "bf16", True, 0, seed=B + 2)
    check_backward(few, 2, 2, d, "bf16", False, 0, seed=B + 3)


def test_gradients_are_the_slopes_of_the_loss():
    """Central differences of the 64-bit loss sum(O dO) along random directions.

    The difference itself is exact to h^2; a gradient G off by at most b(G) elementwise moves
    the slope along X by at most sum(b |X|)."""
    lens, H, Hk, d = [37, 1, 90], 4, 2, 64
    q, k, v, do, cu = make(lens, H, Hk, d, "bf16", 5)
    s = 1 / math.sqrt(d)
    o, lse = fa2.forward_varlen(q, k, v, cu, s, True)
    got = fa2.backward_varlen(q, k, v, o, do, lse, cu, s, True)
    ok()
    _, bound = packed_backward(q, k, v, do, lens, s, True)
    x = [t.double() for t in (q, k, v)]
    h = 1e-4

    def loss(xs):
        at, total = 0, 0.0
        for n in lens:
            for i in range(H):
                sl, g = slice(at, at + n), i // (H // Hk)
                a = s * xs[0][sl, i] @ xs[1][sl, g].T
                a = torch.where(torch.ones_like(a).tril().bool(), a, float("-inf")).softmax(1)
                total = total + float(((a @ xs[2][sl, g]) * do[sl, i].double()).sum())
            at += n
        return total

    g = torch.Generator(device="cuda").manual_seed(6)
    for i in range(3):
        X = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        up = loss([t + h * X if j == i else t for j, t in enumerate(x)])
        dn = loss([t - h * X if j == i else t for j, t in enumerate(x)])
        slope = (up - dn) / (2 * h)
        mine = float((got[i].double() * X).sum())
        room = float((bound[i] * X.abs()).sum()) + 1e-4 * (1 + abs(slope))
        assert abs(mine - slope) <= room


@pytest.mark.parametrize("d", [64, 128])
def test_one_sequence_agrees_with_the_dense_calls(d):
    B, H, N = 3, 4, 300
    q, k, v, do, cu = make([N] * B, H, H, d, "bf16", 7)
    s = 1 / math.sqrt(d)
    dense = [x.reshape(B, N, H, d).transpose(1, 2).contiguous() for x in (q, k, v, do)]
    for causal, window in ((True, 0), (False, 0), (True, 70)):
        o, lse = fa2.forward_varlen(q, k, v, cu, s, causal, window)
        if window:
            o2, lse2 = fa2.forward_window(*dense[:3], s, window)
        else:
            o2, lse2 = fa2.forward(*dense[:3], s, causal)
        _, _, bo, bl = packed_forward(q, k, v, [N] * B, s, causal, window)
        assert_within(o, o2.transpose(1, 2).reshape(o.shape).double(), 2 * bo, "O")
        assert_within(lse, lse2.transpose(0, 1).reshape(lse.shape).double(), 2 * bl, "LSE")
    ok()


def head_major(x):
    """The same [T, heads, d] values stored [heads, T, d]."""
    return x.transpose(0, 1).contiguous().transpose(0, 1)


def test_strides_and_outputs_of_ones_own():
    """Head-major and padded inputs give the bits of contiguous ones; rows behind the last
    sequence and the padding between rows stay as they were, in every output."""
    lens, H, Hk, d, extra = [70, 0, 200, 1], 6, 2, 64, 9
    n = sum(lens)
    q, k, v, do, cu = make(lens, H, Hk, d, "bf16", 8, extra=extra)
    s = 0.1
    with torch.no_grad():
        for t in (q, k, v, do):
            t[n:] = float("nan")
    base = fa2.forward_varlen(*(t.contiguous() for t in (q, k, v)), cu, s, True)
    T = n + extra
    for form in (head_major, lambda x: x):
        buf = torch.full((T, H + 3, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        o = buf[:, 1:H + 1, :d]
        lse = torch.full((H, T), 7.0, device="cuda")
        assert fa2.fa2_fwd_varlen(form(q), form(k), form(v), o, lse, cu, s, True) == fa2.FA2_OK
        ok()
        assert torch.equal(o[:n], base[0][:n]) and torch.equal(lse[:, :n], base[1][:, :n])
        assert (lse[:, n:] == 7).all() and (buf[n:] == 7).all()
        assert (buf[:, 0] == 7).all() and (buf[:, H + 1:] == 7).all() and (buf[:, :, d:] == 7).all()
        outs = [torch.full((T, h + 1, d + 8), 7.0, dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk)]
        views = [x[:, :-1, :d] for x in outs]
        ws = torch.empty(fa2.fa2_bwd_varlen_workspace_size(len(lens), T, H, Hk, d) + 64, dtype=torch.uint8,
                         device="cuda").fill_(255)
        need = ws.numel() - 64
        assert fa2.fa2_bwd_varlen(form(q), form(k), form(v), o, form(do), lse, *views, cu, ws[:need], s,
                                  True) == fa2.FA2_OK
        ok()
        assert (ws[need:] == 255).all()
        ref, bound = packed_backward(q[:n], k[:n], v[:n], do[:n], lens, s, True)
        for x, w, r, b in zip(outs, views, ref, bound):
            assert_within(w[:n], r, b, "gradient")
            assert (x[n:] == 7).all() and (x[:, -1] == 7).all() and (x[:, :, d:] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_sequence_does_not_reach_its_neighbours(d):
    """NaN and infinities all through one sequence leave the others' bits as they were."""
    lens, H, Hk = [130, 77, 300, 5], 4, 2
    q, k, v, do, cu = (t.clone() for t in make(lens, H, Hk, d, "bf16", 9))
    s = 0.1

    def both():
        o, lse = fa2.forward_varlen(q, k, v, cu, s, True)
        return (o, lse.t()) + fa2.backward_varlen(q, k, v, o, do, lse, cu, s, True)

    clean = both()
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[130:207] = False
    for bad in (float("nan"), float("inf"), -float("inf")):
        for t in (q, k, v, do):
            t[130:207] = bad
        dirty = both()
        ok()
        for i, (a, b) in enumerate(zip(clean, dirty)):
            if i == 2:  # dQ is summed by atomics
                assert torch.isfinite(b[keep].float()).all()
                assert (a[keep].float() - b[keep].float()).abs().max() <= 2 ** -7 * a.float().abs().max()
            else:
                assert torch.equal(a[keep], b[keep]), i


def test_repeatable():
    q, k, v, do, cu = make([700, 129, 1, 400], 8, 2, 128, "bf16", 10)
    o, lse = fa2.forward_varlen(q, k, v, cu, 0.08, True)
    g = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.08, True)
    for _ in range(5):
        o2, lse2 = fa2.forward_varlen(q, k, v, cu, 0.08, True)
        g2 = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.08, True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert torch.equal(g[1], g2[1]) and torch.equal(g[2], g2[2])
    ok()


def test_captured_call_follows_the_lengths():
    """Two graphs captured over one workspace and set of buffers, replayed in turn with other
    lengths written to the offsets between."""
    H, Hk, d, T, B = 4, 2, 64, 500, 4
    q, k, v, do, cu = make([T, 0, 0, 0], H, Hk, d, "bf16", 11)
    o, lse = torch.zeros_like(do), torch.zeros((H, T), device="cuda")
    grads = [torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hk, Hk)]
    ws = torch.empty(fa2.fa2_bwd_varlen_workspace_size(B, T, H, Hk, d), dtype=torch.uint8, device="cuda")
    s = 0.125

    def step(stream, causal):
        assert fa2.fa2_fwd_varlen(q, k, v, o, lse, cu, s, causal, 0, stream) == fa2.FA2_OK
        assert fa2.fa2_bwd_varlen(q, k, v, o, do, lse, *grads, cu, ws, s, causal, 0, stream) == fa2.FA2_OK

    step(None, True)
    torch.cuda.synchronize()
    graphs = []
    for causal in (True, False):
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step(st, causal)
        graphs.append(g)
    for lens in ([100, 0, 250, 150], [499, 1, 0, 0], [0, 0, 0, 500]):
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        cu.copy_(torch.tensor(at, dtype=torch.int32))
        for causal, g in zip((True, False), graphs):
            g.replay()
            torch.cuda.synchronize()
            ro, rl, bo, bl = packed_forward(q, k, v, lens, s, causal)
            assert_within(o, ro, bo, "O")
            assert_within(lse, rl, bl, "LSE")
            ref, bound = packed_backward(q, k, v, do, lens, s, causal)
            for x, r, b in zip(grads, ref, bound):
                assert_within(x, r, b, "gradient")
    ok()
    del graphs


def test_two_streams_at_once():
    runs = []
    for i in range(2):
        q, k, v, do, cu = make([300 + i, 90, 1], 4, 2, 64 * (i + 1), "bf16", 12 + i)
        o, lse = fa2.forward_varlen(q, k, v, cu, 0.1, True)
        g = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.1, True)
        runs.append((q, k, v, do, cu, (o, lse) + g[1:], torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        for q, k, v, do, cu, ref, st in runs:
            with torch.cuda.stream(st):
                o, lse = fa2.forward_varlen(q, k, v, cu, 0.1, True)
                g = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.1, True)
                outs.append(((o, lse) + g[1:], ref))
    torch.cuda.synchronize()
    for got, ref in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    ok()


def test_calls_on_a_stream_that_is_not_the_current_one():
    """Outputs and workspace allocated by the call belong to its stream: tensors of their sizes
    that the current stream allocates and fills meanwhile are others."""
    q, k, v, do, cu = make([300, 90, 1, 700], 4, 2, 64, "bf16", 16)
    o, lse = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    g = fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.1, True)
    need = fa2.fa2_bwd_varlen_workspace_size(4, q.shape[0], 4, 2, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(5):
        o2, lse2 = fa2.forward_varlen(q, k, v, cu, 0.1, True, stream=st)
        outs.append((o2, lse2) + fa2.backward_varlen(q, k, v, o2, do, lse2, cu, 0.1, True, stream=st))
        torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.full_like(do, 3)
    st.synchronize()
    for got in outs:
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert torch.equal(got[3], g[1]) and torch.equal(got[4], g[2])
        # dQ: sums of at most six 32-bit partials in another order, then one rounding each
        assert ((got[2].float() - g[0].float()).abs() <= 2 ** -7 * g[0].float().abs() + 1e-5).all()
    ok()


def test_a_window_past_32_bits_hides_nothing():
    q, k, v, _, cu = make([300, 5], 4, 2, 64, "bf16", 17)
    full = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5):
        got = fa2.forward_varlen(q, k, v, cu, 0.1, True, window)
        assert all(torch.equal(a, b) for a, b in zip(got, full))
    ok()


def test_row_offsets_past_32_bits():
    """Rows so far apart that element offsets pass 2^32."""
    H, Hk, d, T = 2, 1, 64, 70000
    buf = torch.zeros((T, 65536), dtype=torch.bfloat16, device="cuda")
    lens = [T - 300, 300]
    g = torch.Generator(device="cuda").manual_seed(13)
    part = buf[T - 300:, :4 * d]
    part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    q = buf[:, :H * d].view(T, H, d)
    k, v = (buf[:, (H + i) * d:(H + i + 1) * d].view(T, Hk, d) for i in range(2))
    o = torch.zeros((T, H, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((H, T), device="cuda")
    cu = torch.tensor([T - 300, T], dtype=torch.int32, device="cuda")
    assert fa2.fa2_fwd_varlen(q, k, v, o, lse, cu, 0.1, True) == fa2.FA2_OK
    ok()
    ro, rl, bo, bl = packed_forward(q[-300:], k[-300:], v[-300:], [300], 0.1, True)
    assert_within(o[-300:], ro, bo, "O")
    assert_within(lse[:, -300:], rl, bl, "LSE")
    assert not o[:-300].any() and not lse[:, :-300].any()


def test_a_batch_of_no_rows():
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    o, lse = fa2.forward_varlen(q, k, k, cu, 0.1, True)
    dq, dk, dv = fa2.backward_varlen(q, k, k, o, o, lse, cu, 0.1, True)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0) and dk.shape == (0, 2, 64)
    q, k, v, do, _ = make([40], 4, 2, 64, "bf16", 14)
    o, lse = torch.full_like(do, 7), torch.full((4, 40), 7.0, device="cuda")
    assert fa2.fa2_fwd_varlen(q, k, v, o, lse, cu, 0.1, True) == fa2.FA2_OK
    ok()
    assert (o == 7).all() and (lse == 7).all()
    grads = [torch.full_like(x, 7).contiguous() for x in (q, k, v)]
    ws = torch.empty(fa2.fa2_bwd_varlen_workspace_size(2, 40, 4, 2, 64), dtype=torch.uint8, device="cuda")
    assert fa2.fa2_bwd_varlen(q, k, v, o, do, lse, *grads, cu, ws, 0.1, True) == fa2.FA2_OK
    ok()
    assert all((x == 7).all() for x in grads)


def test_bad_offsets_stay_inside_the_tensors():
    """Offsets that fall, repeat or leave the tensors: nothing outside is touched (the results
    are unspecified)."""
    q, k, v, do, _ = make([300], 4, 2, 64, "bf16", 15)
    buf = torch.full((302, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    o, lse = buf[1:301], torch.zeros((4, 300), device="cuda")
    for at in ([0, 300, 0, 300], [-5, 100, 2 ** 31 - 1, 40], [290, 20, 300, -2 ** 31], [0, 300, 300, 300]):
        cu = torch.tensor(at, dtype=torch.int32, device="cuda")
        assert fa2.fa2_fwd_varlen(q, k, v, o, lse, cu, 0.1, True) == fa2.FA2_OK
        fa2.backward_varlen(q, k, v, o, do, lse, cu, 0.1, True)
        ok()
        assert (buf[0] == 7).all() and (buf[301] == 7).all()
