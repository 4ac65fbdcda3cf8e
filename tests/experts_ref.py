"""Plain 64-bit forms of the router and the experts' products, and bounds on what the library's
rounding may change.

The bounds count roundings.  A sum of m fp32 terms, in any order, is off by at most
(m + 16) * 2^-23 * sum|terms| (one rounding or truncation, below 2^-23 relative, per addition
and scale); the result is then rounded once to the token type (half a step:
2^-8 bf16, 2^-11 fp16, relative, and 2^-25 absolute below fp16's normal range).

fp8 codes meet in matrix instructions that add eight consecutive products at a time and cut each
product, towards zero, at 2^-13 of the group's largest power of two 2^E (measured: beside
products +2^16 and -2^16, a third of 2^3 survives and one of 2^2 vanishes, in the
same eight elements only).  The largest product is at least 2^E, so a product loses less than
2^-13 * max|product of the eight| and the eight lose less than 2^-10 of it; with
max|x w| <= max|x| * max|w| the row loses less than 2^-10 * sum over the eights of
max|x| * max|w|, which is `cut` below.
"""
import math

import torch

F32_STEP = 2.0 ** -23
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def pack_counts(counts, W):
    """(ep_recv_count [W][L*W], recv_offsets [W+1]) of rows per expert (all from source 0..W-1
    in turn), as dispatch lays them out, and the experts' row ranges."""
    E = len(counts)
    per = torch.zeros((E, W), dtype=torch.int64)
    for e, c in enumerate(counts):
        for s in range(W):
            per[e, s] = c // W + (1 if s < c % W else 0)
    ranks = per.view(W, E // W * W)
    erc = ranks.cumsum(1).to(torch.int32)
    off = torch.zeros(W + 1, dtype=torch.int64)
    off[1:] = ranks.sum(1).cumsum(0)
    ends = torch.tensor(counts).cumsum(0).tolist()
    return erc, off, list(zip([0] + ends[:-1], ends))


def power(b):
    return torch.pow(torch.tensor(2.0, dtype=torch.float64, device=b.device), b.double() - 127)


def codes_to_f64(c, scales):
    v = c.double()
    if scales is None:
        return v
    if scales.dtype == torch.uint8:
        return v * power(scales).repeat_interleave(32, -1)
    return v * scales.double().unsqueeze(-1)


def w4_to_f64(w, scales, kind, group):
    lo, hi = (w & 15).long(), (w >> 4).long()
    u = torch.stack((lo, hi), -1).flatten(-2)
    if kind == "int4":
        v, s = torch.where(u > 7, u - 16, u).double(), scales.double()
    else:
        v = torch.tensor(E2M1, dtype=torch.float64, device=w.device)[u]
        s = power(scales)
    return v * s.repeat_interleave(group, -1)


def _eights(v):
    """Largest magnitude of each eight consecutive elements."""
    return v.abs().view(*v.shape[:-1], -1, 8).amax(-1)


def product(x, w, ranges, swiglu, surplus=None, cut=False):
    """(S or its SwiGLU, bound before the last rounding) of fp64 rows x [R][I] and weights
    w [E][N][I].  surplus [E][N][I] (optional): magnitude of what is added and taken away again
    per element of x (in place of |w| in the bound).  cut: fp8 instructions."""
    R, I = x.shape
    N = w.shape[1]
    half = N // 2
    y = torch.zeros((R, half if swiglu else N), dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(ranges):
        if lo == hi:
            continue
        s = x[lo:hi] @ w[e].t()
        mag = x[lo:hi].abs() @ (w[e].abs() if surplus is None else surplus[e]).t()
        d = (I + 16) * F32_STEP * mag
        if cut:
            d = d + 2.0 ** -10 * (_eights(x[lo:hi]) @ _eights(w[e]).t())
        if swiglu:
            g, u, dg, du = s[:, :half], s[:, half:], d[:, :half], d[:, half:]
            silu = g / (1 + torch.exp(-g))
            y[lo:hi] = silu * u
            # |silu'| < 1.1; the fp32 exponential and division are within 2^-17 for |g| < 100
            err[lo:hi] = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -17 * y[lo:hi].abs()
        else:
            y[lo:hi], err[lo:hi] = s, d
    return y, err


def check(out, y, err, rows):
    assert torch.isfinite(out[:rows].float()).all()
    diff = (out[:rows].double() - y).abs()
    tol = err + HALF_STEP[out.dtype] * (y.abs() + err) + (
        2.0 ** -25 if out.dtype == torch.float16 else 2.0 ** -134)
    bad = diff > tol
    assert not bad.any(), (int(bad.sum()), float((diff / tol).max()))


def gate(logits, bias, K, sigmoid, groups, keep, top, renorm, factor):
    """Ids and weights of fp64 definitions, one token at a time."""
    T, n = logits.shape
    z = logits.double()
    score = torch.sigmoid(z) if sigmoid else torch.softmax(z, 1)
    choice = score if bias is None else score + bias.double()
    order = z if bias is None else choice
    part = choice if top == 2 else order
    ids = torch.zeros((T, K), dtype=torch.int32)
    weights = torch.zeros((T, K), dtype=torch.float64)
    size = n // groups
    for t in range(T):
        stay = set(range(n))
        if groups > 1:
            vals = []
            for g in range(groups):
                m = sorted(part[t, g * size:(g + 1) * size].tolist(), reverse=True)
                vals.append(sum(m[:top]))
            kept = sorted(range(groups), key=lambda g: (-vals[g], g))[:keep]
            stay = {i for g in kept for i in range(g * size, (g + 1) * size)}
        o = order[t].tolist()
        best = sorted(stay, key=lambda i: (-o[i], i))[:K]
        w = [float(score[t, i]) for i in best]
        if renorm:
            total = math.fsum(w) + 1e-20
            w = [v / total for v in w]
        ids[t] = torch.tensor(best, dtype=torch.int32)
        weights[t] = torch.tensor([v * factor for v in w], dtype=torch.float64)
    return ids, weights
