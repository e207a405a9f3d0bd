"""Measured cases of the packed and paged attention operators.

Five operators that a model runs on batches of requests of different lengths:

  varlen_fwd   attention over packed sequences (grouped heads), output and log-sum-exp
  varlen_bwd   its gradient with respect to the queries, keys and values
  paged        attention of each request's new tokens over its paged key/value cache
  tables       block tables, slots and positions of a step, from the requests' lengths
  append       the step's new keys and values written into the paged cache

Where ``own`` is false ``run`` computes them from elementary torch operations in
32 bits, on sequences padded to the longest; where it is true it makes the calls
of the library.  ``exact`` computes them sequence by sequence in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
NEG = float("-inf")


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # three short prompts at once: the call's latency
        {"name": "varlen_fwd_short", "op": "varlen_fwd", "batch": 3, "longest": 90, "heads": 8,
         "kv_heads": 2, "head_dim": 64, "dtype": "fp16", "window": 0, "mix": 1},
        # a usual batch of prompts, an empty one and one of a single token among them
        {"name": "varlen_fwd_batch", "op": "varlen_fwd", "batch": 12, "longest": 2048, "heads": 16,
         "kv_heads": 8, "head_dim": 64, "dtype": "bf16", "window": 0, "mix": 2},
        # long prompts, four query heads to a key/value head
        {"name": "varlen_fwd_long", "op": "varlen_fwd", "batch": 4, "longest": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "window": 0, "mix": 3},
        # a training step's packed documents, head dim 64
        {"name": "varlen_bwd_batch", "op": "varlen_bwd", "batch": 8, "longest": 1024, "heads": 16,
         "kv_heads": 4, "head_dim": 64, "dtype": "bf16", "window": 0, "mix": 4},
        # the same with longer documents and head dim 128
        {"name": "varlen_bwd_long", "op": "varlen_bwd", "batch": 6, "longest": 4096, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "dtype": "bf16", "window": 0, "mix": 5},
        # a decode step of a few requests with short caches: latency
        {"name": "paged_decode_few", "op": "paged", "batch": 4, "context": 700, "chunk": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16", "window": 0,
         "mix": 6},
        # a decode step of a full batch with long caches: bandwidth
        {"name": "paged_decode_full", "op": "paged", "batch": 64, "context": 8192, "chunk": 1,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16", "window": 0,
         "mix": 7},
        # chunks of prompts over what is cached of them, a decode step and an idle request beside
        {"name": "paged_chunks", "op": "paged", "batch": 6, "context": 8192, "chunk": 1024,
         "heads": 32, "kv_heads": 4, "head_dim": 128, "block": 64, "dtype": "bf16", "window": 0,
         "mix": 8},
        # a decode step's tables: one token more for each request
        {"name": "tables_decode", "op": "tables", "batch": 64, "context": 8192, "chunk": 1,
         "block": 16, "mix": 9},
        # the tables of many prompts and chunks at once
        {"name": "tables_prompts", "op": "tables", "batch": 500, "context": 1024, "chunk": 2048,
         "block": 16, "mix": 10},
        # the keys and values of a decode step
        {"name": "append_decode", "op": "append", "batch": 64, "context": 700, "chunk": 1,
         "kv_heads": 8, "head_dim": 128, "block": 16, "dtype": "bf16", "mix": 11},
        # those of a batch of long prompts
        {"name": "append_prompts", "op": "append", "batch": 12, "context": 1024, "chunk": 8192,
         "kv_heads": 8, "head_dim": 128, "block": 64, "dtype": "bf16", "mix": 12},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["varlen_fwd", "varlen_bwd", "paged", "paged", "tables", "append"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 8])
    c = {"op": op, "mix": rng.randrange(1 << 20)}
    if op in ("varlen_fwd", "varlen_bwd", "paged"):
        if kv * group > 32:
            group = 4
        c.update(heads=kv * group, kv_heads=kv, head_dim=rng.choice([40, 64, 64, 96, 128, 128]),
                 dtype=rng.choice(["bf16", "bf16", "fp16"]), window=0)
    if op in ("varlen_fwd", "varlen_bwd"):
        c["longest"] = _log_uniform(rng, 20, 8000 if op == "varlen_fwd" else 4000)
        # at most what the longest listed cases hold
        most = max(1, int((4 if op == "varlen_fwd" else 1.4) * (8192 / c["longest"]) ** 2))
        c["batch"] = min(most, _log_uniform(rng, 1, 60))
        if rng.random() < 0.25:
            c["window"] = _log_uniform(rng, 1, c["longest"])
    elif op == "paged":
        c["block"] = rng.choice([8, 16, 32, 64, 128])
        c["context"] = _log_uniform(rng, 16, 8000)
        c["chunk"] = 1 if rng.random() < 0.5 else _log_uniform(rng, 2, 1000)
        c["batch"] = _log_uniform(rng, 1, 60 if c["chunk"] == 1 else 6)
        if rng.random() < 0.2:
            c["window"] = _log_uniform(rng, 16, 4000)
    else:
        c["block"] = rng.choice([8, 16, 32, 64, 128])
        c["context"] = _log_uniform(rng, 1, 8000 if op == "tables" else 1000)
        c["chunk"] = 1 if rng.random() < 0.4 else _log_uniform(rng, 2, 2000)
        c["batch"] = _log_uniform(rng, 1, 400 if op == "tables" else 30)
        if op == "append":
            c.update(kv_heads=kv, head_dim=rng.choice([40, 64, 96, 128]),
                     dtype=rng.choice(["bf16", "fp16"]))
    return c


def _lengths(rng, batch, longest):
    """Lengths of a ragged batch: the longest first, then 30 to 100 % of it; batches of six and
    more hold a request of one token and one of none."""
    n = [longest] + [max(1, int(longest * rng.uniform(0.3, 1.0))) for _ in range(batch - 1)]
    if batch >= 6:
        n[2], n[4] = 1, 0
    return n


def _shape(case):
    """(new tokens, cached tokens) of each request."""
    rng = random.Random(case["mix"])
    if case["op"].startswith("varlen"):
        return _lengths(rng, case["batch"], case["longest"]), None
    context = _lengths(rng, case["batch"], case["context"])
    if case["chunk"] == 1:
        return [1] * case["batch"], context
    return _lengths(rng, case["batch"], case["chunk"])[::-1], context


def _pairs(new, context, window):
    """(query, key) pairs of one head and keys that any query sees, causal."""
    pairs = keys = 0
    for b, n in enumerate(new):
        c = context[b] if context else 0
        if n == 0:
            continue
        if window:
            lo = max(0, c + 1 - window)  # first key that the first query sees
            keys += c + n - lo
            full = max(0, min(n, window - c))  # queries that see every key up to their own
            pairs += full * c + full * (full + 1) // 2 + (n - full) * window
        else:
            keys += c + n
            pairs += n * c + n * (n + 1) // 2
    return pairs, keys


def work(case):
    new, context = _shape(case)
    T, B = sum(new), len(new)
    if case["op"] in ("varlen_fwd", "varlen_bwd", "paged"):
        H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
        pairs, keys = _pairs(new, context, case["window"])
    if case["op"] == "varlen_fwd":
        return {"flops": 4 * H * d * pairs, "bytes": 2 * T * d * (2 * H + 2 * Hk) + 4 * T * H + 4 * B + 4}
    if case["op"] == "varlen_bwd":
        return {"flops": 10 * H * d * pairs, "bytes": 2 * T * d * (4 * H + 4 * Hk) + 4 * T * H + 4 * B + 4}
    if case["op"] == "paged":
        return {"flops": 4 * H * d * pairs,
                "bytes": 4 * keys * Hk * d + 4 * T * H * d + 4 * T * H + 4 * (keys // case["block"]) + 8 * B + 4}
    if case["op"] == "tables":
        bs = case["block"]
        had = sum(-(-c // bs) for c in context)
        need = sum(-(-(c + n) // bs) for c, n in zip(context, new))
        # lengths in, free blocks in, table entries out, offsets and lengths out, two numbers a token out
        return {"flops": 0, "bytes": 8 * B + 8 * (need - had) + 8 * B + 4 + 8 * T + 4}
    return {"flops": 0, "bytes": 8 * T * case["kv_heads"] * case["head_dim"] + 4 * T}


# ------------------------------------------------------------------ the inputs

def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    new, context = _shape(case)
    T, B = sum(new), len(new)
    s = dict(case)
    s.update(T=T, B=B, longest_new=max(new))
    ints = dict(device="cuda", dtype=torch.int32)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, **ints)
    if case["op"].startswith("varlen"):
        H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
        dt = DTYPES[case["dtype"]]
        # queries, keys and values lie side by side, as one projection writes them
        qkv = _randn(gen, (T, H + 2 * Hk, d), dt)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hk], v=qkv[:, H + Hk:], scale=d ** -0.5)
        if case["op"] == "varlen_bwd":
            s["do"] = _randn(gen, (T, H, d), dt)
            # what the forward call left: the rounded output and the log-sum-exp
            o, lse = _plain_varlen_fwd(s)
            s.update(o=o, lse=lse)
        return s
    bs = case["block"]
    need = [-(-(c + n) // bs) for c, n in zip(context, new)]
    had = [-(-c // bs) for c in context]
    blocks = sum(need) + 8
    ids = torch.randperm(blocks, generator=gen, device="cuda").to(torch.int32)
    most = max(need) + 2
    col = torch.arange(most, device="cuda")
    use = torch.tensor(need if case["op"] != "tables" else had, device="cuda")
    first = torch.cumsum(use, 0) - use
    table = torch.where(col < use[:, None], ids[(first[:, None] + col).clamp(max=blocks - 1)].long(), 0).to(torch.int32)
    s.update(table=table, context_lens=torch.tensor(context, **ints), new_lens=torch.tensor(new, **ints),
             seq_lens=torch.tensor([c + n for c, n in zip(context, new)], **ints), most=most, blocks=blocks)
    if case["op"] == "tables":
        s["free"] = ids[sum(had):].contiguous()
        return s
    Hk, d, dt = case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    if case["op"] == "paged":
        s["q"] = _randn(gen, (T, case["heads"], d), dt)
        s["scale"] = d ** -0.5
        s["k_cache"] = _randn(gen, (blocks, Hk, bs, d), dt)
        s["v_cache"] = _randn(gen, (blocks, Hk, bs, d), dt)
        return s
    kv = _randn(gen, (T, 2 * Hk, d), dt)
    s.update(k=kv[:, :Hk], v=kv[:, Hk:])
    s["k_cache"] = torch.zeros((blocks, Hk, bs, d), dtype=dt, device="cuda")
    s["v_cache"] = torch.zeros((blocks, Hk, bs, d), dtype=dt, device="cuda")
    t = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    pos = s["context_lens"].long()[seq] + t - s["cu"].long()[seq]
    s["slots"] = (table[seq, pos // bs].long() * bs + pos % bs).to(torch.int32)
    return s


# ------------------------------------------------------------------ the plain forms

def _padded(cu, longest, T):
    """Row of the packed tensor for each (sequence, position), and which of them exist."""
    at = cu[:-1, None].long() + torch.arange(longest, device=cu.device)
    real = at < cu[1:, None].long()
    return at.clamp(max=max(T - 1, 0)), real


def _spread(x, at, heads):
    """Packed [T, heads * g, d] as [B, heads, g * L, d] in 32 bits (rows: g, then position)."""
    B, L = at.shape
    T, H, d = x.shape
    return x.float()[at].view(B, L, heads, H // heads, d).permute(0, 2, 3, 1, 4).reshape(B, heads, -1, d)


def _gather(y, at, real, T, shape):
    """The reverse of _spread: padded [B, heads, g * L, d] back to packed rows."""
    B, L = at.shape
    heads, d = y.shape[1], y.shape[3]
    rows = y.view(B, heads, -1, L, d).permute(0, 3, 1, 2, 4).reshape(B * L, -1, d)
    out = torch.zeros((T + 1, rows.shape[1], d), dtype=y.dtype, device=y.device)
    out[torch.where(real, at, T).reshape(-1)] = rows
    return out[:T].reshape(shape)


def _hidden(q_pos, k_pos, q_real, k_real, window):
    """[B, 1, L, Lk]: the keys that a query does not see."""
    far = q_pos[:, :, None] - k_pos[:, None, :]
    hide = (far < 0) | ~k_real[:, None, :] | ~q_real[:, :, None]
    if window:
        hide = hide | (far >= window)
    return hide[:, None]


def _softmax(s, hide, group):
    """(P not yet divided, its row sums, log-sum-exp) of scores s [B, heads, g * L, Lk], in place.
    A row that sees nothing has zeros and -inf."""
    B, heads, rows, Lk = s.shape
    s = s.view(B, heads * group, rows // group, Lk).masked_fill_(hide, NEG).view(B, heads, rows, Lk)
    m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == NEG, torch.zeros_like(m), m)
    p = s.sub_(m0).exp_()
    l = p.sum(-1, keepdim=True)
    return p, l, (m0 + l.log())


def _plain_varlen_fwd(s):
    H, Hk = s["heads"], s["kv_heads"]
    at, real = _padded(s["cu"], s["longest_new"], s["T"])
    pos = torch.arange(at.shape[1], device=at.device).expand(at.shape)
    q, k, v = (_spread(s[n], at, Hk) for n in "qkv")
    p, l, lse = _softmax((q * s["scale"]) @ k.transpose(-1, -2), _hidden(pos, pos, real, real, s["window"]), H // Hk)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    o = _gather(o, at, real, s["T"], s["q"].shape).to(s["q"].dtype)
    lse = _gather(lse, at, real, s["T"], (s["T"], H)).t().contiguous()
    return o, lse


def _plain_varlen_bwd(s):
    H, Hk, T = s["heads"], s["kv_heads"], s["T"]
    at, real = _padded(s["cu"], s["longest_new"], T)
    pos = torch.arange(at.shape[1], device=at.device).expand(at.shape)
    q, k, v, do, o = (_spread(s[n], at, Hk) for n in ("q", "k", "v", "do", "o"))
    hide = _hidden(pos, pos, real, real, s["window"])
    g = H // Hk
    lse = _spread(s["lse"].t()[:, :, None], at, Hk)
    p = (q * s["scale"]) @ k.transpose(-1, -2)
    p = p.sub_(lse).exp_().view(*hide.shape[:1], H, *hide.shape[2:]).masked_fill_(hide, 0.0).view(p.shape)
    # rows past a sequence's end are other rows' copies: they take no part
    real_q = real[:, None, None, :, None].expand(-1, Hk, g, -1, 1).reshape(at.shape[0], Hk, -1, 1)
    do = torch.where(real_q, do, torch.zeros_like(do))
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = (ds @ k) * s["scale"]
    dk = (ds.transpose(-1, -2) @ q) * s["scale"]
    return tuple(_gather(x, at, real, T, s[n].shape).to(s[n].dtype) for x, n in ((dq, "q"), (dk, "k"), (dv, "v")))


def _plain_paged(s):
    H, Hk, T, bs = s["heads"], s["kv_heads"], s["T"], s["block"]
    at, real = _padded(s["cu"], s["longest_new"], T)
    B, n = s["table"].shape

    def cached(c):
        return c[s["table"].long()].permute(0, 2, 1, 3, 4).reshape(B, Hk, n * bs, -1).float()

    q, k, v = _spread(s["q"], at, Hk), cached(s["k_cache"]), cached(s["v_cache"])
    k_pos = torch.arange(n * bs, device=at.device).expand(B, -1)
    k_real = k_pos < s["seq_lens"][:, None]
    q_pos = s["context_lens"][:, None] + torch.arange(at.shape[1], device=at.device)
    p, l, lse = _softmax((q * s["scale"]) @ k.transpose(-1, -2), _hidden(q_pos, k_pos, real, k_real, s["window"]), H // Hk)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    o = _gather(o, at, real, T, s["q"].shape).to(s["q"].dtype)
    lse = _gather(lse, at, real, T, (T, H)).t().contiguous()
    return o, lse


def _plain_tables(s):
    bs, T = s["block"], s["T"]
    ctx, new = s["context_lens"].long(), s["new_lens"].long()
    total = ctx + new
    cu = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    had, need = (ctx + bs - 1) // bs, (total + bs - 1) // bs
    take = need - had
    first = torch.cumsum(take, 0) - take
    col = torch.arange(s["table"].shape[1], device=ctx.device)
    fresh = (col >= had[:, None]) & (col < need[:, None])
    pick = (first[:, None] + col - had[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][pick], s["table"])
    t = torch.arange(T, device=ctx.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    pos = ctx[seq] + t - cu[seq]
    slots = table[seq, pos // bs].long() * bs + pos % bs
    as_int = torch.int32
    return table, cu.to(as_int), total.to(as_int), pos.to(as_int), slots.to(as_int), take.sum().to(as_int).reshape(1)


def _plain_append(s):
    slot = s["slots"].long()
    block, row = slot // s["block"], slot % s["block"]
    s["k_cache"][block, :, row] = s["k"]
    s["v_cache"][block, :, row] = s["v"]
    return s["k_cache"], s["v_cache"]


PLAIN = {"varlen_fwd": _plain_varlen_fwd, "varlen_bwd": _plain_varlen_bwd, "paged": _plain_paged,
         "tables": _plain_tables, "append": _plain_append}


def run(state):
    s = state
    if not own:
        return PLAIN[s["op"]](s)
    from exact_io_aware_74_b200 import fa2
    if s["op"] == "varlen_fwd":
        return fa2.forward_varlen(s["q"], s["k"], s["v"], s["cu"], s["scale"], True, window=s["window"])
    if s["op"] == "varlen_bwd":
        return fa2.backward_varlen(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], s["cu"], s["scale"], True,
                                   window=s["window"])
    if s["op"] == "paged":
        return fa2.forward_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["seq_lens"], s["scale"],
                                 True, window=s["window"])
    if s["op"] == "tables":
        return fa2.paged_tables(s["context_lens"], s["new_lens"], s["free"], s["table"], s["T"], s["block"])
    return fa2.paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])


# ------------------------------------------------------------------ the definition, in 64 bits

def _exact_sequence(q, k, v, scale, offset, window):
    """Probabilities, output and log-sum-exp of one sequence and key/value head: queries
    [g, n, d] at positions offset .. offset + n - 1, keys and values [m, d] at 0 .. m - 1."""
    n, m = q.shape[1], k.shape[0]
    i = torch.arange(n, device=q.device)[:, None] + offset
    j = torch.arange(m, device=q.device)[None, :]
    sees = j <= i
    if window:
        sees = sees & (j > i - window)
    x = torch.einsum("gid,jd->gij", q, k) * scale
    x = torch.where(sees, x, torch.full((), NEG, dtype=x.dtype, device=x.device))
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[..., None])
    return p, torch.einsum("gij,jd->gid", p, v), lse


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    new, context = _shape(case)
    if case["op"] == "append":
        out = []
        for x, c in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            rows = c.double().transpose(1, 2).reshape(-1, *x.shape[1:])
            rows[s["slots"].long()] = x.double()
            out.append(rows.view(c.shape[0], c.shape[2], *x.shape[1:]).transpose(1, 2).contiguous())
        return out
    H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    g, T, bs = H // Hk, s["T"], case.get("block", 0)
    f64 = dict(device="cuda", dtype=torch.float64)
    o, lse = torch.zeros((T, H, d), **f64), torch.full((H, T), NEG, **f64)
    grads = [torch.zeros((T, h, d), **f64) for h in (H, Hk, Hk)] if case["op"] == "varlen_bwd" else None
    row = 0
    for b, n in enumerate(new):
        if n == 0:
            continue
        here = slice(row, row + n)
        row += n
        for h in range(Hk):
            heads = slice(h * g, (h + 1) * g)
            q = s["q"][here, heads].double().transpose(0, 1)
            if case["op"] == "paged":
                total = context[b] + n
                ids = s["table"][b, :-(-total // bs)].long()
                k, v = (s[c][ids, h].double().reshape(-1, d)[:total] for c in ("k_cache", "v_cache"))
                offset = context[b]
            else:
                k, v = s["k"][here, h].double(), s["v"][here, h].double()
                offset = 0
            # a few query heads at a time: the score rows are kept whole
            step = max(1, min(g, int(4e9 // (8 * n * k.shape[0] + 1))))
            for a in range(0, g, step):
                qa, ha = q[a:a + step], slice(h * g + a, h * g + min(a + step, g))
                p, oa, la = _exact_sequence(qa, k, v, s["scale"], offset, case["window"])
                o[here, ha] = oa.transpose(0, 1)
                lse[ha, here] = la
                if grads:
                    do = s["do"][here, ha].double().transpose(0, 1)
                    dp = torch.einsum("gid,jd->gij", do, v)
                    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
                    grads[0][here, ha] = torch.einsum("gij,jd->gid", ds, k).transpose(0, 1)
                    grads[1][here, h] += torch.einsum("gij,gid->jd", ds, qa)
                    grads[2][here, h] += torch.einsum("gij,gid->jd", p, do)
    return tuple(grads) if grads else (o, lse)
