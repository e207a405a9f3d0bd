"""Packed batches of the sizes at which the order and the cut of the work items change, against
the 64-bit reference of packed_ref.py.

The library makes an item of every 128-key tile (backward) or block of query tiles (forward) of
every sequence and key/value head.  By the number of items it takes one or two query tiles to a
forward item, cuts the backward's key tiles into parts, and puts the heads into groups that
follow one another; by the number of sequences it keeps their lengths at hand or not.
"""

import random

import pytest

from test_varlen_gpu import MODES, check_backward, check_forward

pytestmark = pytest.mark.gpu


def lengths(n, longest, seed):
    r = random.Random(seed)
    return [r.choice([longest, longest - 1, r.randrange(longest), 1, 0]) if i % 5 == 0 else
            r.randrange(longest // 2, longest) for i in range(n)]


@pytest.mark.parametrize("causal,window", MODES)
@pytest.mark.parametrize("H,Hk,d", [(4, 4, 64), (4, 4, 128), (6, 2, 96)])
def test_forward_of_two_query_tiles(H, Hk, d, causal, window):
    """148 blocks of two query tiles and more: 16 sequences of up to 1000 tokens."""
    lens = [700] * 14 + [1000, 0, 263]
    blocks = sum(-(-n // (256 // (H // Hk))) for n in lens) * Hk
    assert blocks >= 148
    check_forward(lens, H, Hk, d, "bf16", causal, window, seed=d)


@pytest.mark.parametrize("causal,window", MODES)
@pytest.mark.parametrize("d", [64, 128])
def test_backward_of_whole_key_tiles(d, causal, window):
    """More than 444 key tiles, none cut, of at most 96 sequences."""
    lens = [700] * 39 + [1] + [130]
    assert sum(-(-n // 128) for n in lens) * 2 > 444 and len(lens) <= 96
    check_backward(lens, 4, 2, d, "bf16", causal, window, seed=d)


@pytest.mark.parametrize("B", [250, 300], ids=["held", "not-held"])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_forward_of_several_head_groups(B, d):
    """1776 blocks and more of 11 heads: groups of 4, 4 and 3 (250 sequences), or 3, 3, 3 and 2."""
    check_forward(lengths(B, 40, B + d), 11, 11, d, "bf16", True, 0, seed=B)


@pytest.mark.parametrize("B", [95, 120], ids=["held", "not-held"])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_of_several_head_groups(B, d):
    """1184 key tiles and more of 7 or 8 heads: groups that the heads do not fill evenly."""
    lens = lengths(B, 260, B + d)
    for H, Hk in ((8, 8), (14, 7)):
        assert (sum(lens) // 128 + B) * Hk >= 1184
        check_backward(lens, H, Hk, d, "bf16", True, 0, seed=B)
    check_backward(lens, 8, 8, d, "fp16", False, 0, seed=B + 1)
    check_backward(lens, 8, 8, d, "bf16", True, 60, seed=B + 2)
