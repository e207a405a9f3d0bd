"""Bounded waits of the packed and paged kernels: a load that never comes (test hook) ends in
FA2_ERR_TIMEOUT from a wait of the right kernel, and the context stays usable."""

import pytest
import torch

from exact_io_aware_74_b200 import fa2

pytestmark = pytest.mark.gpu


@pytest.fixture
def missing_load():
    fa2.fa2_debug_set(1, 50)
    yield
    fa2.fa2_debug_set(0, 0)


def _packed(lens, d, H=4, Hk=2):
    g = torch.Generator(device="cuda").manual_seed(1)
    T = sum(lens)
    q, k, v = (torch.randn((T, h, d), generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hk, Hk))
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return q, k, v, cu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[300, 20], [1000] * 60], ids=["few", "many"])
def test_packed_forward(d, lens, missing_load):
    q, k, v, cu = _packed(lens, d)
    fa2.forward_varlen(q, k, v, cu, 0.1, True)
    rc, site = fa2.fa2_get_device_status()
    assert rc == fa2.FA2_ERR_TIMEOUT and 80 <= site < 100
    fa2.fa2_debug_set(0, 0)
    a = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    b = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)
    assert all(torch.equal(x, y) for x, y in zip(a, b)) and torch.isfinite(a[0].float()).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[300, 20], [700] * 40], ids=["few", "many"])
def test_packed_backward(d, lens):
    q, k, v, cu = _packed(lens, d)
    o, lse = fa2.forward_varlen(q, k, v, cu, 0.1, True)
    ref = fa2.backward_varlen(q, k, v, o, q, lse, cu, 0.1, True)
    fa2.fa2_debug_set(1, 50)
    try:
        fa2.backward_varlen(q, k, v, o, q, lse, cu, 0.1, True)
        rc, site = fa2.fa2_get_device_status()
    finally:
        fa2.fa2_debug_set(0, 0)
    assert rc == fa2.FA2_ERR_TIMEOUT and 100 <= site < 118
    got = fa2.backward_varlen(q, k, v, o, q, lse, cu, 0.1, True)
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])


@pytest.mark.parametrize("new", [1, 200])
def test_paged(new, missing_load):
    H, Hk, d, block = 8, 2, 128, 16
    kc = torch.randn((200, Hk, block, d), device="cuda").to(torch.bfloat16)
    q = torch.randn((2 * new, H, d), device="cuda").to(torch.bfloat16)
    ints = dict(dtype=torch.int32, device="cuda")
    table = torch.arange(180, **ints).view(2, 90)
    cu, lens = torch.tensor([0, new, 2 * new], **ints), torch.tensor([1400, 900], **ints)
    fa2.forward_paged(q, kc, kc, table, cu, lens, 0.1, True)
    rc, site = fa2.fa2_get_device_status()
    assert rc == fa2.FA2_ERR_TIMEOUT and 80 <= site < 100
    fa2.fa2_debug_set(0, 0)
    a, b = (fa2.forward_paged(q, kc, kc, table, cu, lens, 0.1, True) for _ in range(2))
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
