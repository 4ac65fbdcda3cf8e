"""The router with enough tokens for four of them to share a wave (4096, up to 576 ids, 16 groups),
and just below, against the 64-bit form in whole tensors."""
import math

import pytest
import torch

import combine_quant_amd as cq

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _expected(z, K, sigmoid, groups, keep):
    """Ids and weights without a bias, groups by their best logit: all by 64-bit tensors."""
    T, n = z.shape
    z = z.double()
    score = torch.sigmoid(z) if sigmoid else torch.softmax(z, 1)
    order = z
    if groups > 1:
        best = z.view(T, groups, n // groups).amax(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :keep]
        off = torch.ones((T, groups), dtype=torch.bool).scatter_(1, kept, False)
        order = z.masked_fill(off.repeat_interleave(n // groups, 1), -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :K]
    return ids, torch.gather(score, 1, ids)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("W,BS,E,Z,K,groups,keep", [
    (8, 512, 256, 0, 8, 8, 4), (16, 257, 16, 0, 3, 1, 1), (16, 259, 512, 4, 16, 1, 1), (9, 456, 180, 1, 16, 1, 1),
    (8, 512, 64, 0, 8, 16, 5), (16, 300, 576, 0, 9, 16, 5), (16, 256, 576, 1, 16, 1, 1), (10, 410, 30, 0, 2, 3, 1),
    (8, 511, 256, 0, 8, 8, 3), (16, 300, 256, 0, 12, 64, 20),
])
@pytest.mark.parametrize("spread", ["random", "ties", "equal"])
def test_many_tokens(W, BS, E, Z, K, groups, keep, sigmoid, spread):
    n = E + Z
    g = torch.Generator().manual_seed(W + K)
    z = torch.randn((W * BS, n), generator=g) * 2
    if spread == "ties":
        z = (z * 4).round() / 4
    elif spread == "equal":
        z[:] = 0.5
        z[::3] = torch.randn((len(z[::3]), n), generator=g)
        z[1::3, ::2] = -math.inf
    cfg = cq.make_config(W, E, BS, 1024, K, zero_expert_num=Z)
    ids, w = cq.gate_topk(cfg, cq.make_gate(cq.MOE_SCORE_SIGMOID if sigmoid else cq.MOE_SCORE_SOFTMAX, groups, keep),
                          z.view(W, BS, n).to(DEV))
    rid, rw = _expected(z, K, sigmoid, groups, keep)
    assert torch.equal(ids.view(-1, K).cpu().long(), rid)
    # the score, within 2^-24.8 (the softmax sum's exponentials) and an fp32 rounding
    diff = (w.view(-1, K).cpu().double() - rw).abs()
    assert (diff <= 2.0 ** -23 * rw + 2.0 ** -149).all()
