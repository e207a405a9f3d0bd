"""64-bit reference of attention over packed sequences and paged caches, with the error
bounds the GPU results are held to.

Everything is computed sequence by sequence from whole score rows in float64.  With
u = finfo(dtype).eps / 2 the half step of the 16-bit type:

* O.  The weights P are rounded to 16 bits and O is their weighted mean, so numerator
  and denominator each move by at most u (relative): 2 u sum_j P |v|.  The exponentials
  and the 32-bit scores add a relative error of the weights below w = 2^-19 (1 + max |s|)
  (the score's 32-bit sum is off by at most about d 2^-24 of sum |q k| scale, which the
  tests' inputs keep below 2^-19 max |s|-like terms).  Storing O adds u |O|.  In fp16 a weight
  below 2^-14 is subnormal: off by at most 2^-25 each, with a largest weight of at
  least 1: 2^-25 sum_j |v|.  A stored result below 2^-14 is subnormal too: the step there is
  2^-24, so that storing any result moves it by at most max(u |x|, 2^-25).
* LSE.  Sums of up to 2^15 positive 32-bit terms and one logarithm: 2e-5 + 2^-20 max |s|.
* dV = P^T dO with P rounded: (u + w) sum_i P |dO| + u |dV|.
* dS = P (dP - D) rounded; D = rowsum(dO o) uses the stored O, off by its own bound:
  |err dS| <= (u + w) |dS| + P dD + 2^-19 P (|dO| |v|), dD = sum |dO| bound(O).  dQ and dK
  carry that through K and Q, plus u of themselves.  In fp16 dS below 2^-14 is off by at
  most 2^-25 each.
"""

import torch


def _bounds_of(dtype):
    u = torch.finfo(dtype).eps / 2
    return u, (2.0 ** -25 if dtype == torch.float16 else 0.0)


def visible(n, m, offset, causal, window, device):
    i = torch.arange(n, device=device)[:, None] + offset
    j = torch.arange(m, device=device)[None, :]
    see = torch.ones((n, m), dtype=torch.bool, device=device)
    if causal:
        see = j <= i
        if window:
            see = see & (j > i - window)
    return see


def forward_one(q, k, v, scale, offset, causal, window, dtype):
    """q [n,d], k, v [m,d] float64.  Returns O, LSE, bound(O), bound(LSE), P."""
    n, m = q.shape[0], k.shape[0]
    u, sub = _bounds_of(dtype)
    if m == 0:
        z = torch.zeros_like(q)
        inf = torch.full((n,), float("-inf"), dtype=q.dtype, device=q.device)
        return z, inf, z, torch.zeros_like(inf), q.new_zeros((n, 0))
    see = visible(n, m, offset, causal, window, q.device)
    s = torch.where(see, scale * (q @ k.T), float("-inf"))
    any_key = see.any(1)
    smax = torch.where(see, s, torch.zeros_like(s)).abs().amax(1)
    top = torch.where(any_key, s.amax(1), torch.zeros_like(smax))
    e = torch.exp(s - top[:, None])
    l = e.sum(1)
    p = e / torch.where(any_key, l, torch.ones_like(l))[:, None]
    lse = torch.where(any_key, top + torch.log(l), float("-inf"))
    o = p @ v
    w = 2.0 ** -19 * (1 + smax)[:, None]
    bo = (2 * u + w) * (p @ v.abs()) + u * o.abs() + sub + sub * (see.double() @ v.abs()) + 1e-9
    bl = 2e-5 + 2.0 ** -20 * smax
    return o, lse, bo, bl, p


def backward_one(q, k, v, do, scale, offset, causal, window, dtype):
    """Gradients of one sequence and query head, and their bounds."""
    u, sub = _bounds_of(dtype)
    o, _, bo, _, p = forward_one(q, k, v, scale, offset, causal, window, dtype)
    see = visible(q.shape[0], k.shape[0], offset, causal, window, q.device)
    smax = torch.where(see, scale * (q @ k.T), q.new_zeros(())).abs().amax(1)
    w = 2.0 ** -19 * (1 + smax)[:, None]
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdim=True))
    eds = (u + w) * ds.abs() + p * (do.abs() * bo).sum(1, keepdim=True) + \
        2.0 ** -19 * p * (do.abs() @ v.abs().T) + sub * see.double()
    dv = p.T @ do
    bv = ((u + w) * p + sub * see.double()).T @ do.abs() + u * dv.abs() + sub + 1e-9
    dq, dk = scale * (ds @ k), scale * (ds.T @ q)
    bq = scale * (eds @ k.abs()) + u * dq.abs() + sub + 1e-9
    bk = scale * (eds.T @ q.abs()) + u * dk.abs() + sub + 1e-9
    return (dq, dk, dv), (bq, bk, bv)


def packed_forward(q, k, v, lens, scale, causal, window=0, caches=None):
    """q [T,H,d], k, v [T,Hkv,d] (or ``caches``: per sequence float64 k, v [m,Hkv,d]).
    Returns O, LSE [H,T] and their bounds over the rows of the sequences."""
    T, H, d = q.shape
    dtype, dev = q.dtype, q.device
    f = dict(dtype=torch.float64, device=dev)
    o, bo = torch.zeros((T, H, d), **f), torch.zeros((T, H, d), **f)
    lse, bl = torch.zeros((H, T), **f), torch.zeros((H, T), **f)
    row = 0
    for b, n in enumerate(lens):
        if caches is None:
            kb, vb = k[row:row + n].double(), v[row:row + n].double()
        else:
            kb, vb = caches[b]
        g = H // kb.shape[1]
        for h in range(H):
            if n == 0:
                continue
            r = forward_one(q[row:row + n, h].double(), kb[:, h // g], vb[:, h // g], scale,
                            kb.shape[0] - n, causal, window, dtype)
            o[row:row + n, h], lse[h, row:row + n], bo[row:row + n, h], bl[h, row:row + n] = r[:4]
        row += n
    return o, lse, bo, bl


def packed_backward(q, k, v, do, lens, scale, causal, window=0):
    """dQ, dK, dV of the packed forward, and their bounds."""
    H, Hk = q.shape[1], k.shape[1]
    g = H // Hk
    outs = [torch.zeros(x.shape, dtype=torch.float64, device=q.device) for x in (q, k, v)]
    errs = [torch.zeros_like(x) for x in outs]
    row = 0
    for n in lens:
        at = slice(row, row + n)
        for h in range(H if n else 0):
            gr, er = backward_one(q[at, h].double(), k[at, h // g].double(), v[at, h // g].double(),
                                  do[at, h].double(), scale, 0, causal, window, q.dtype)
            for i, c in enumerate((h, h // g, h // g)):
                outs[i][at, c] += gr[i]
                errs[i][at, c] += er[i]
        row += n
    return outs, errs


def assert_within(got, ref, bound, what):
    got = got.double()
    same_inf = torch.isinf(ref) & (got == ref)
    off = torch.where(same_inf, torch.zeros_like(bound), (got - ref).abs())
    assert torch.isfinite(off).all(), f"{what}: not finite"
    over = off - bound
    i = int(over.argmax()) if over.numel() else 0
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{what}: off by {float(off.flatten()[i]):.3g}, bound {float(bound.flatten()[i]):.3g} at {i}"
