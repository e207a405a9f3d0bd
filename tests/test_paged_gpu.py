"""Paged caches: tables from lengths, the write into the cache and attention over it, each
against a plain implementation, and a run of them together.

Bounds of the attention: see packed_ref.py.  Tables and writes are exact.
"""

import math
import random

import pytest
import torch

from exact_io_aware_74_b200 import fa2
from packed_ref import assert_within, packed_forward

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ok():
    assert fa2.fa2_get_device_status() == (fa2.FA2_OK, 0)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Step:
    """A cache of random blocks in random order, and a step's queries over it."""

    def __init__(self, context, new, H, Hk, d, block, dtype, seed, layout="heads", spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.context, self.new, self.block, self.scale = context, new, block, 1 / math.sqrt(d)
        self.total = [c + n for c, n in zip(context, new)]
        need = [-(-t // block) for t in self.total]
        blocks = sum(need) + spare
        most = max(need + [1]) + 1
        order = torch.randperm(blocks, generator=g, device="cuda").tolist()
        # entries past a request's blocks hold what no cache has
        self.table = torch.full((len(new), most), -12345, dtype=torch.int32)
        for b, n in enumerate(need):
            self.table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        self.table = self.table.cuda()
        shape = {"heads": (blocks, Hk, block, d), "rows": (blocks, block, Hk, d),
                 "both": (blocks, 2, Hk, block, d)}[layout]
        if layout == "both":  # keys and values of a block side by side
            kv = torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda")
            self.k_cache, self.v_cache = kv[:, 0], kv[:, 1]
        else:
            kv = [torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2)]
            self.k_cache, self.v_cache = kv if layout == "heads" else (t.transpose(1, 2) for t in kv)
        self.caches = []
        for b, t in enumerate(self.total):
            k, v = (torch.randn((t, Hk, d), generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
            for cache, x in ((self.k_cache, k), (self.v_cache, v)):
                for i in range(need[b]):
                    part = x[i * block:(i + 1) * block]
                    cache[int(self.table[b, i]), :, :part.shape[0]] = part.transpose(0, 1)
            self.caches.append((k.double(), v.double()))
        T = sum(new)
        self.q = torch.randn((T, H, d), generator=g, device="cuda").to(DT[dtype])
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu, self.lens = ints(cu), ints(self.total)

    def run(self, causal=True, window=0, **kw):
        r = fa2.forward_paged(self.q, self.k_cache, self.v_cache, self.table, self.cu, self.lens, self.scale,
                              causal, window, **kw)
        ok()
        return r

    def check(self, causal=True, window=0):
        o, lse = self.run(causal, window)
        ro, rl, bo, bl = packed_forward(self.q, None, None, self.new, self.scale, causal, window, self.caches)
        assert_within(lse, rl, bl, "LSE")
        assert_within(o, ro, bo, "O")


BATCHES = [([0], [1]), ([1], [1]), ([5, 127, 128, 0], [1, 1, 1, 1]), ([1000, 17, 300], [1, 1, 1]),
           ([0, 0, 0], [130, 1, 300]), ([100, 0, 257, 3, 640], [20, 0, 129, 1, 7]), ([4000], [3]),
           ([2000, 30], [500, 1])]


@pytest.mark.parametrize("context,new", BATCHES, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hk", [(8, 2), (3, 3)])
def test_attention(context, new, d, H, Hk):
    s = Step(context, new, H, Hk, d, 16, "bf16", seed=sum(context) + d + H)
    s.check()
    s.check(False)
    s.check(True, 1)
    s.check(True, 90)


@pytest.mark.parametrize("block", [8, 16, 32, 64, 128, 256, 384])
@pytest.mark.parametrize("layout", ["heads", "rows", "both"])
def test_blocks_and_layouts(block, layout):
    Step([0, 700, 129, 20], [300, 1, 5, 0], 8, 2, 64, block, "bf16", seed=block, layout=layout).check()
    Step([777, 1], [1, 1], 8, 1, 128, block, "fp16", seed=block + 1, layout=layout).check()


@pytest.mark.parametrize("d", [8, 24, 72, 96, 136, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_head_dims(d, dtype):
    Step([300, 40], [1, 1], 6, 2, d, 16, dtype, seed=d).check()
    Step([300, 0, 9], [140, 33, 1], 4, 4, d, 32, dtype, seed=d + 1).check()


@pytest.mark.parametrize("H,Hk", [(1, 1), (7, 1), (20, 4), (65, 1), (128, 1), (32, 8)])
def test_head_groups(H, Hk):
    Step([300, 1500, 0], [1, 1, 1], H, Hk, 128, 16, "bf16", seed=H).check()
    Step([300, 10], [70, 3], H, Hk, 64, 64, "bf16", seed=H + 1).check(True, 100)


@pytest.mark.parametrize("H,Hk", [(16, 1), (17, 1), (24, 1), (64, 2)])
@pytest.mark.parametrize("d,dtype", [(64, "bf16"), (64, "fp16"), (128, "bf16"), (128, "fp16")])
def test_rows_of_single_tokens(H, Hk, d, dtype):
    """Decode steps with as many rows to an item as its forms hold, or just more."""
    Step([300, 1500, 0, 127], [1, 1, 1, 1], H, Hk, d, 16, dtype, seed=H + d).check()
    Step([900, 3], [2, 2], H, Hk, d, 64, dtype, seed=H + d + 1).check(True, 200)


def test_many_requests():
    r = random.Random(3)
    n = 300
    Step([r.randrange(400) for _ in range(n)], [r.choice([0, 1, 1, 1, 2]) for _ in range(n)], 4, 1, 64, 16, "bf16",
         seed=4).check()
    for n in (256, 257, 600):  # about as many as a scheduling warp keeps the counts of
        new = [r.choice([0, 1, 5]) for _ in range(n)]
        new[n // 2] = 200
        Step([r.randrange(60) for _ in range(n)], new, 4, 2, 64, 16, "bf16", seed=n).check()
    Step([r.randrange(3000) for _ in range(40)], [1] * 40, 8, 4, 128, 16, "bf16", seed=5).check()


def test_one_request_with_a_long_cache():
    Step([32000], [1], 8, 1, 128, 64, "bf16", seed=6).check()
    Step([20000, 5], [9, 1], 4, 2, 64, 16, "fp16", seed=7).check()


def test_more_queries_than_keys():
    """A request whose queries reach further back than its keys: the first rows see none."""
    s = Step([0, 40], [60, 5], 4, 2, 64, 16, "bf16", seed=8)
    s.lens = ints([20, 3])
    o, lse = s.run()
    caches = [(k[:m], v[:m]) for (k, v), m in zip(s.caches, (20, 3))]
    ro, rl, bo, bl = packed_forward(s.q, None, None, s.new, s.scale, True, 0, caches)
    assert_within(o, ro, bo, "O")
    assert_within(lse, rl, bl, "LSE")
    assert not o[:40].any() and (lse[:, :40] == float("-inf")).all()
    assert not o[60:62].any()
    s.lens = ints([0, 0])
    for causal in (True, False):
        o, lse = s.run(causal)
        assert not o.any() and (lse == float("-inf")).all()


@pytest.mark.parametrize("n", [1, 9, 40, 700])
@pytest.mark.parametrize("d", [64, 256])
def test_requests_without_keys_between_others(n, d):
    """Many blocks of rows that see no key, between requests that have keys."""
    s = Step([100, 0, 0, 0, 0, 200, 0], [1, n, n, n, n, 2, n], 4, 2, d, 16, "bf16", seed=n)
    s.lens = ints([101, 0, 0, 0, 0, 202, 0])
    caches = [(k[:m], v[:m]) for (k, v), m in zip(s.caches, (101, 0, 0, 0, 0, 202, 0))]
    for causal in (True, False):
        o, lse = s.run(causal)
        ro, rl, bo, bl = packed_forward(s.q, None, None, s.new, s.scale, causal, 0, caches)
        assert_within(o, ro, bo, "O")
        assert_within(lse, rl, bl, "LSE")


def test_rows_behind_the_last_sequence_and_the_workspace_end():
    s = Step([100, 300], [1, 20], 8, 2, 128, 16, "bf16", seed=9)
    T = 21
    ref = s.run()
    q = torch.cat([s.q, torch.full((7, 8, 128), float("nan"), dtype=s.q.dtype, device="cuda")])
    o, lse = torch.full_like(q, 7), torch.full((8, T + 7), 7.0, device="cuda")
    need = fa2.fa2_fwd_paged_workspace_size(2, T + 7, 8, 2, 128)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    assert fa2.fa2_fwd_paged(q, s.k_cache, s.v_cache, o, lse, s.table, s.cu, s.lens, ws[:need], s.scale,
                             True) == fa2.FA2_OK
    ok()
    ro, rl, bo, bl = packed_forward(s.q, None, None, s.new, s.scale, True, 0, s.caches)
    assert_within(o[:T], ro, bo, "O")
    assert_within(lse[:, :T], rl, bl, "LSE")
    assert ref[0].shape == (T, 8, 128)
    assert (o[T:] == 7).all() and (lse[:, T:] == 7).all() and (ws[need:] == 255).all()


def test_blocks_outside_the_cache_are_reported():
    """They read as zeros, say so, and leave the other requests' results alone."""
    s = Step([300, 200, 100], [1, 2, 1], 8, 2, 64, 16, "bf16", seed=10)
    ro, rl, bo, bl = packed_forward(s.q, None, None, s.new, s.scale, True, 0, s.caches)
    for bad in (-1, s.k_cache.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = s.table.clone()
        table[1, 3] = bad
        o, lse = fa2.forward_paged(s.q, s.k_cache, s.v_cache, table, s.cu, s.lens, s.scale, True)
        rc, site = fa2.fa2_get_device_status()
        assert rc == fa2.FA2_ERR_INVALID_ARG and site == 120
        k, v = (x.clone() for x in s.caches[1])
        k[48:64], v[48:64] = 0, 0
        z = packed_forward(s.q, None, None, s.new, s.scale, True, 0, [s.caches[0], (k, v), s.caches[2]])
        assert_within(o, z[0], z[2], "O")
        assert_within(lse, z[1], z[3], "LSE")
    s.check()


@pytest.mark.parametrize("new", [[1, 1, 1], [40, 300, 7]])
def test_bad_offsets_stay_inside_the_tensors(new):
    """Offsets that fall, repeat or leave the tensors, and lengths of any sign: nothing outside the
    outputs is touched (the results are unspecified)."""
    s = Step([200, 0, 500], new, 4, 2, 64, 16, "bf16", seed=32)
    T = s.q.shape[0]
    s.table.clamp_(0)  # entries that a wrong length may reach
    buf = torch.full((T + 2, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4 * T + 2,), 7.0, device="cuda")
    ws = torch.empty(fa2.fa2_fwd_paged_workspace_size(3, T, 4, 2, 64), dtype=torch.uint8, device="cuda")
    top = 2 ** 31 - 1
    for at, lens in (([0, T, 0, T], [200, 500, 90]), ([-5, 1, top, 2], [1, top, 30]), ([T, 0, T, -top - 1], [60] * 3),
                     ([0, T, T, T], [-7, -top - 1, top])):
        assert fa2.fa2_fwd_paged(s.q, s.k_cache, s.v_cache, buf[1:T + 1], lse[1:-1].view(4, T), s.table, ints(at),
                                 ints(lens), ws, s.scale, True) == fa2.FA2_OK
        ok()
        assert (buf[0] == 7).all() and (buf[T + 1] == 7).all() and lse[0] == 7 and lse[-1] == 7
    s.check()


def test_repeatable():
    s = Step([5000, 129, 0, 2000], [1, 1, 1, 1], 16, 4, 128, 16, "bf16", seed=11)
    o, lse = s.run()
    for _ in range(5):
        o2, lse2 = s.run()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_block_offsets_past_32_bits():
    """A cache whose element offsets pass 2^32: 10 GB of keys and as much of values."""
    Hk, block, d, blocks = 8, 64, 128, 80000
    kc, vc = (torch.zeros((blocks, Hk, block, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(12)
    ids = [blocks - 1, 3, 65540]
    k, v = (torch.randn((130, Hk, d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = ints([ids[i // block] * block + i % block for i in range(130)])
    fa2.paged_append(k, v, kc, vc, slots)
    q = torch.randn((2, 16, d), generator=g, device="cuda").to(torch.bfloat16)
    o, lse = fa2.forward_paged(q, kc, vc, ints([ids]), ints([0, 2]), ints([130]), 0.09, True)
    ok()
    ro, rl, bo, bl = packed_forward(q, None, None, [2], 0.09, True, 0, [(k.double(), v.double())])
    assert_within(o, ro, bo, "O")
    assert_within(lse, rl, bl, "LSE")


# ------------------------------------------------------------------ tables

def plain_tables(context, new, free, table, T, block):
    table = [list(r) for r in table]
    positions, slots, cu, k = [], [], [0], 0
    for b, (c, n) in enumerate(zip(context, new)):
        had, need = -(-c // block), -(-(c + n) // block)
        for i in range(had, need):
            if i < len(table[b]):
                table[b][i] = free[k] if k < len(free) else -1
            elif k < len(free):
                pass
            k += 1
        for p in range(c, c + n):
            e = table[b][p // block] if p // block < len(table[b]) else -1
            positions.append(p)
            slots.append(e * block + p % block if e >= 0 else -1)
        cu.append(cu[-1] + n)
    positions, slots = positions[:T], slots[:T]
    positions += [0] * (T - len(positions))
    slots += [-1] * (T - len(slots))
    return table, cu, [c + n for c, n in zip(context, new)], positions, slots, [k]


@pytest.mark.parametrize("B", [1, 2, 31, 300, 513, 1500])
@pytest.mark.parametrize("block", [1, 16, 100])
@pytest.mark.parametrize("short,room", [(0, 0), (5, 0), (0, 40), (0, -7)])
def test_tables(B, block, short, room):
    """``short``: blocks missing from the free list; ``room``: of T beside the step's tokens."""
    r = random.Random(B * 1000 + block + short + room)
    context = [r.choice([0, 1, 15, 16, 17, r.randrange(500)]) for _ in range(B)]
    new = [r.choice([0, 1, 1, 2, 16, r.randrange(300)]) for _ in range(B)]
    most = max(1, max(-(-(c + n) // block) for c, n in zip(context, new)) - (1 if B == 31 else 0))
    wanted = sum(-(-(c + n) // block) - -(-c // block) for c, n in zip(context, new))
    free = list(range(10 ** 6, 10 ** 6 + max(0, wanted - short)))
    table = [[r.randrange(1000) for _ in range(most)] for _ in range(B)]
    T = max(0, sum(new) + room)
    ref = plain_tables(context, new, free, table, T, block)
    got = fa2.paged_tables(ints(context), ints(new), ints(free), ints(table), T, block)
    ok()
    for name, x, y in zip(("table", "cu", "lens", "positions", "slots", "used"), got, ref):
        assert x.tolist() == y, name


def test_tables_count_negative_lengths_as_none():
    got = fa2.paged_tables(ints([-3, 5]), ints([2, -9]), ints([8, 9]), ints([[0, 0], [4, 0]]), 3, 4)
    ok()
    assert [x.tolist() for x in got] == [[[8, 0], [4, 0]], [0, 2, 2], [2, 5], [0, 1, 0], [32, 33, -1], [1]]


def test_tables_of_lengths_up_to_31_bits():
    """Lengths whose rounding up to whole blocks passes 2^31; the table keeps what it held."""
    top = 2 ** 31 - 1
    for context, new in (([top - 20, 5], [20, 3]), ([top, 0], [0, 9]), ([top - 3, top], [3, 0])):
        for block in (16, 1, 1000):
            table = [[7, 8], [9, 10]]
            free = list(range(100, 120))
            got = fa2.paged_tables(ints(context), ints(new), ints(free), ints(table), sum(new) + 2, block)
            ok()
            taken = -(-(context[0] + new[0]) // block) - -(-context[0] // block)
            for i in range(-(-context[1] // block), min(2, -(-(context[1] + new[1]) // block))):
                k = taken + i - -(-context[1] // block)
                table[1][i] = free[k] if k < len(free) else -1
            assert got[0].tolist() == table
            assert got[2].tolist() == [c + n for c, n in zip(context, new)]
            at = [c + i for c, n in zip(context, new) for i in range(n)]
            assert got[3].tolist() == at + [0, 0]
            assert got[4].tolist()[:new[0]] == [-1] * new[0] and got[4].tolist()[-2:] == [-1, -1]


def test_tables_of_sums_past_31_bits_stay_inside():
    """The results are unspecified; nothing outside the tables is touched."""
    top = 2 ** 31 - 1
    for context, new in (([0, 0, 0], [top, top, top]), ([top, top, 5], [top, 9, top]), ([1, 2, 3], [2 ** 30] * 3)):
        buf = ints([[7] * 4] * 5)
        out = ints([7] * 12)
        positions, slots = ints([7] * 12), ints([7] * 12)
        assert fa2.fa2_paged_tables(ints(context), ints(new), ints([1, 2, 3]), buf[1:4], out[1:5], out[6:9],
                                    positions[1:11], slots[1:11], out[10:11], 16) == fa2.FA2_OK
        ok()
        assert (buf[0] == 7).all() and (buf[4] == 7).all()
        assert [int(out[i]) for i in (0, 5, 9, 11)] == [7] * 4
        assert [int(x[i]) for x in (positions, slots) for i in (0, 11)] == [7] * 4


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("T", [1, 7, 300])
@pytest.mark.parametrize("Hk,d,block", [(1, 8, 1), (2, 64, 16), (8, 128, 16), (3, 256, 24), (1, 72, 64)])
@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_append(T, Hk, d, block, layout):
    g = torch.Generator(device="cuda").manual_seed(T + d)
    blocks = -(-T // block) + 4
    shape = (blocks, Hk, block, d) if layout == "heads" else (blocks, block, Hk, d)
    caches = [torch.randn(shape, generator=g, device="cuda").to(torch.float16) for _ in range(2)]
    views = [c if layout == "heads" else c.transpose(1, 2) for c in caches]
    before = [v.clone() for v in views]
    kv = torch.randn((T, 2 * Hk + 1, d), generator=g, device="cuda").to(torch.float16)
    k, v = kv[:, :Hk], kv[:, Hk + 1:]
    slots = torch.randperm(blocks * block, generator=g, device="cuda")[:T].to(torch.int32)
    slots[T // 2] = -1
    fa2.paged_append(k, v, *views, slots)
    ok()
    for x, old, now in zip((k, v), before, views):
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                old[s // block, :, s % block] = x[t]
        assert torch.equal(old, now)


def test_append_reports_slots_outside_the_cache():
    kc, vc = (torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    for bad in (64, 2 ** 31 - 1):
        fa2.paged_append(k, k, kc, vc, ints([1, bad, 63]))
        assert fa2.fa2_get_device_status() == (fa2.FA2_ERR_INVALID_ARG, 121)
        assert int(kc.ne(0).sum()) == int(vc.ne(0).sum()) == 2 * 2 * 64
    ok()


# ------------------------------------------------------------------ together

def _serve(steps, H, Hk, d, block, window, graph):
    """Requests that grow step by step: tables, append, attention.  Every step's output is that
    of attention over the whole sequences so far."""
    g = torch.Generator(device="cuda").manual_seed(20)
    B, blocks, most, room = len(steps[0]), 64, 24, max(sum(s) for s in steps)
    kc, vc = (torch.full((blocks, Hk, block, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    pool = torch.full_like(free, -1)
    context, new = ints([0] * B), ints([0] * B)
    q = torch.zeros((room, H, d), dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros((room, Hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    o, lse = torch.zeros_like(q), torch.zeros((H, room), device="cuda")
    ws = torch.empty(fa2.fa2_fwd_paged_workspace_size(B, room, H, Hk, d), dtype=torch.uint8, device="cuda")
    cu, lens, used = ints([0] * (B + 1)), ints([0] * B), ints([0])
    positions, slots = ints([0] * room), ints([0] * room)
    s = d ** -0.5

    def step(stream=None):
        assert fa2.fa2_paged_tables(context, new, pool, table, cu, lens, positions, slots, used, block,
                                    stream) == fa2.FA2_OK
        assert fa2.fa2_paged_append(k, v, kc, vc, slots, stream) == fa2.FA2_OK
        assert fa2.fa2_fwd_paged(q, kc, vc, o, lse, table, cu, lens, ws, s, True, window, stream) == fa2.FA2_OK

    run = step
    if graph:
        step()
        torch.cuda.synchronize()
        st, cg = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=st):
            step(st)
        run = cg.replay
    taken, history = 0, [[] for _ in range(B)]
    for lengths in steps:
        new.copy_(ints(lengths))
        pool.fill_(-1)
        pool[:blocks - taken].copy_(free[taken:])
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        run()
        torch.cuda.synchronize()
        ok()
        taken += int(used)
        at = 0
        for b, n in enumerate(lengths):
            history[b].append((k[at:at + n].double(), v[at:at + n].double()))
            at += n
        caches = [tuple(torch.cat([h[i] for h in hs]) for i in range(2)) for hs in history]
        assert lens.tolist() == [c[0].shape[0] for c in caches]
        ro, rl, bo, bl = packed_forward(q[:at], None, None, lengths, s, True, window, caches)
        assert_within(o[:at], ro, bo, "O")
        assert_within(lse[:, :at], rl, bl, "LSE")
        context.copy_(lens)


STEPS = [[70, 1, 0, 33], [1, 1, 130, 1], [1, 1, 1, 1], [1, 0, 1, 40], [3, 1, 1, 1]]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("H,Hk,d,block,window", [(8, 2, 64, 16, 0), (4, 4, 128, 32, 0), (6, 1, 96, 16, 50)])
def test_serving_steps(H, Hk, d, block, window, graph):
    _serve(STEPS, H, Hk, d, block, window, graph)


def test_steps_on_a_stream_that_is_not_the_current_one():
    """A call on a given stream, its outputs and workspace allocated by it, while the current
    stream allocates and fills tensors of the same sizes."""
    s = Step([3000, 700, 0, 90], [1, 40, 130, 1], 8, 2, 128, 16, "bf16", seed=30)
    ref = s.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    need = fa2.fa2_fwd_paged_workspace_size(4, s.q.shape[0], 8, 2, 128)
    for stream in (st, st.cuda_stream):
        outs = []
        for _ in range(6):
            outs.append(fa2.forward_paged(s.q, s.k_cache, s.v_cache, s.table, s.cu, s.lens, s.scale, True,
                                          stream=stream))
            torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            torch.full_like(s.q, 3)
        st.synchronize()
        for o, lse in outs:
            assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])
    ok()


def test_a_window_past_32_bits_hides_nothing():
    s = Step([300, 5], [1, 70], 4, 2, 64, 16, "bf16", seed=31)
    full = s.run()
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5):
        got = s.run(True, window)
        assert all(torch.equal(a, b) for a, b in zip(got, full))


def test_prompts_through_the_cache_agree_with_the_packed_forward():
    """Whole prompts written to the cache and read back are the packed prompts."""
    lens, H, Hk, d, block = [200, 1, 77], 8, 2, 128, 16
    s = Step([0] * 3, lens, H, Hk, d, block, "bf16", seed=21)
    k, v = (torch.cat([c[i] for c in s.caches]).to(torch.bfloat16) for i in range(2))
    o1, l1 = s.run()
    o2, l2 = fa2.forward_varlen(s.q, k, v, s.cu, s.scale, True)
    ok()
    _, _, bo, bl = packed_forward(s.q, k, v, lens, s.scale, True)
    assert_within(o1, o2.double(), 2 * bo, "O")
    assert_within(l1, l2.double(), 2 * bl, "LSE")
