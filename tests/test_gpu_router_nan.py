"""Groups without a value (a NaN among their best choices) rank below groups of -infinity, in every
kernel of the router."""
import math

import pytest
import torch

import combine_quant_amd as cq

pytestmark = pytest.mark.gpu

DEV = "cuda"
INF, NAN = math.inf, math.nan


def _value(choices, top):
    """(rank class, sum) of a group: NaN ranks below every number, among its choices and as a
    sum."""
    best = sorted(choices, key=lambda c: (0, 0.0) if math.isnan(c) else (1, c), reverse=True)[:top]
    total = sum(best)
    return (0, 0.0) if math.isnan(total) else (1, total)


def _expected(order, choice, K, groups, keep, top):
    """Ids of one token: order is what ids are compared by, choice what groups are."""
    n = len(order)
    size = n // groups
    values = [_value(choice[g * size:(g + 1) * size], top) for g in range(groups)]
    kept = sorted(range(groups), key=lambda g: (-values[g][0], -values[g][1], g))[:keep]
    stay = [i for g in kept for i in range(g * size, (g + 1) * size)]
    return sorted(stay, key=lambda i: (math.isnan(order[i]), 0 if math.isnan(order[i]) else -order[i], i))[:K]


def _rows(groups, size):
    """Rows whose groups hold each of these, in turn and in both orders."""
    kinds = [[NAN] * size, [-INF] * size, [1.0] + [NAN] * (size - 1), [-INF, NAN] * (size // 2),
             [2.0] + [-INF] * (size - 1), [0.5] * size]
    rows = []
    for shift in range(len(kinds)):
        for step in (1, 5):
            rows.append([v for g in range(groups) for v in kinds[(shift + step * g) % len(kinds)]])
    for a in range(4):                                               # two kinds alone
        for b in range(4):
            rows.append([v for g in range(groups) for v in kinds[a if g % 2 == 0 else b]])
    return torch.tensor(rows)


@pytest.mark.parametrize("groups,size", [(4, 16), (8, 32), (6, 10), (3, 128)])
@pytest.mark.parametrize("repeat", [1, 130, 260])                    # a wave a token, and four
@pytest.mark.parametrize("keep", [1, 2])
def test_by_the_best_logit(groups, size, repeat, keep):
    z = _rows(groups, size)
    T = len(z)
    W, BS, K = 2, T * repeat // 2, 4
    while BS > 512:
        W, BS = W * 2, BS // 2
    cfg = cq.make_config(W, groups * size // W * W, BS, 1024, K, zero_expert_num=groups * size % W)
    assert W * BS == T * repeat
    ids, w = cq.gate_topk(cfg, cq.make_gate(cq.MOE_SCORE_SIGMOID, groups, keep, 1, True),
                          z.repeat(repeat, 1).view(W, BS, -1).to(DEV))
    want = [_expected(r, r, K, groups, keep, 1) for r in z.tolist()]
    assert torch.equal(ids.view(repeat, T, K).cpu(), torch.tensor(want, dtype=torch.int32).expand(repeat, T, K))


@pytest.mark.parametrize("groups,size", [(4, 16), (8, 32), (6, 10), (3, 128)])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("keep", [1, 2])
def test_with_a_bias(groups, size, top, keep):
    """The rows become biases, one token at a time: each choice is the bias or a NaN score."""
    for r in _rows(groups, size).tolist():
        n = groups * size
        special = n % 2
        cfg = cq.make_config(2, n - special, 1, 1024, 4, zero_expert_num=special)
        z = torch.zeros((2, 1, n))
        z[..., [math.isnan(v) for v in r]] = NAN
        bias = torch.tensor([0.0 if math.isnan(v) else v for v in r])
        ids, w = cq.gate_topk(cfg, cq.make_gate(cq.MOE_SCORE_SIGMOID, groups, keep, top, True),
                              z.to(DEV), bias.to(DEV))
        choice = [NAN if math.isnan(v) else 0.5 + v for v in r]
        want = _expected(choice, choice, 4, groups, keep, top)
        assert ids.view(2, 4).tolist() == [want, want], r


@pytest.mark.parametrize("groups,size", [(4, 16), (8, 32), (6, 10), (3, 128)])
@pytest.mark.parametrize("keep", [1, 2])
def test_by_sums_of_scores(groups, size, keep):
    z = _rows(groups, size)
    special = groups * size % 2
    cfg = cq.make_config(2, groups * size - special, len(z) // 2, 1024, 4, zero_expert_num=special)
    ids, w = cq.gate_topk(cfg, cq.make_gate(cq.MOE_SCORE_SIGMOID, groups, keep, 2, True),
                          z.view(2, len(z) // 2, -1).to(DEV))
    score = torch.sigmoid(z.double()).tolist()
    want = [_expected(r, s, 4, groups, keep, 2) for r, s in zip(z.tolist(), score)]
    assert ids.view(-1, 4).tolist() == want
