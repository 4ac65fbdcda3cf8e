"""Plain 64-bit form of the experts' layer of a few tokens, and a bound on what its roundings change.

Bound, counting roundings: gate and up sums of H terms are off by (H + 16) * 2^-23 * sum|terms| at
most, SwiGLU by 2^-17 of its value more (experts_ref.product); the weight's sum and product add 18 *
2^-24, counted as 2^-19; h is then rounded to the token type (half a step).  y sums at most K * F
products, 32 partial sums, K copies and the shared row: (K * F + K + 34) * 2^-23 * sum|terms|; it is
rounded once.
"""
import torch

import block_ref as blk
import experts_ref as ref


def weights(w, scales, parts):
    return w.double() if scales is None else blk.weights_f64(w, scales, parts)


def layer(cfg, x, ids, weight, up, down, mask=None, shared=None):
    """(y, bound before y's rounding) of fp64 x [T][H], up [E][2F][H] and down [E][H][F]."""
    T, K, H, E = cfg.ep_world_size * cfg.bs, cfg.topk, cfg.hidden, cfg.moe_expert_num
    F, half = down.shape[2], ref.HALF_STEP[cq_token(cfg)]
    tiny = 2.0 ** -25 if half == 2.0 ** -11 else 2.0 ** -134
    ids, weight = ids.view(T, K).long(), weight.view(T, K).double()
    if mask is not None:
        on = mask.bool().view(T, -1).expand(T, K)
        ids = torch.where(on, ids, torch.full_like(ids, -1))
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    mag, err = torch.zeros_like(y), torch.zeros_like(y)
    for e in range(E):
        hit = ids == e
        t = torch.nonzero(hit.any(1)).flatten()
        if len(t) == 0:
            continue
        w = (weight * hit).sum(1)[t][:, None]
        s, d = x[t] @ up[e].t(), (H + 16) * ref.F32_STEP * (x[t].abs() @ up[e].abs().t())
        g, u, dg, du = s[:, :F], s[:, F:], d[:, :F], d[:, F:]
        silu = g / (1 + torch.exp(-g))
        h = w * silu * u
        eh = w.abs() * (1.1 * dg * (u.abs() + du) + silu.abs() * du) + (2.0 ** -17 + 2.0 ** -19) * h.abs()
        eh = eh + half * (h.abs() + eh) + tiny
        y[t] += h @ down[e].t()
        err[t] += eh @ down[e].abs().t()
        mag[t] += (h.abs() + eh) @ down[e].abs().t()
    first_copy = E + cfg.zero_expert_num
    copies = ((ids >= first_copy) & (ids < first_copy + cfg.copy_expert_num)) * weight
    y += copies.sum(1, keepdim=True) * x
    mag += copies.abs().sum(1, keepdim=True) * x.abs()
    if shared is not None:
        y += shared.double().view(T, H)
        mag += shared.double().view(T, H).abs()
    return y, err + (K * F + K + 34) * ref.F32_STEP * mag


def cq_token(cfg):
    import combine_quant_amd as cq
    return cq.token_torch_dtype(cfg)
