"""int4 weights with bf16 rows: the codes enter exactly, so nothing is left over from codes of 0,
finite rows near the type's largest value stay finite, and a row's bytes do not depend on how many
other rows its expert has."""
import math

import pytest
import torch

import combine_quant_amd as cq
import experts_ref as ref
from experts_path import path

pytestmark = pytest.mark.gpu

DEV = "cuda"
# experts, ranks, tokens a rank, picks, weight rows: sizes of each kernel
SHAPES = {"stream": (4, 2, 80, 4, 70), "small": (32, 2, 64, 8, 700), "tiles": (32, 2, 256, 8, 770)}


def _config(shape):
    E, W, BS, K, N = SHAPES[shape]
    cfg = cq.make_config(W, E, BS, 1024, K)
    assert path("bf16", cfg, N, False, "int4") == shape
    return cfg, N


def _run(cfg, counts, x, w, ws, group):
    erc, off, ranges = ref.pack_counts(counts, cfg.W)
    mm = cq.make_matmul(x.shape[1], w.shape[1], weight_dtype=cq.MOE_W4_INT4, group_size=group)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))
    torch.cuda.synchronize()
    return out, ranges


def _counts(E, *first):
    return list(first) + [0] * (E - len(first))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_codes_of_zero_give_zero(shape, group):
    cfg, N = _config(shape)
    I = 3 * group
    g = torch.Generator(device=DEV).manual_seed(group)
    counts = _counts(cfg.E, 20, 100, 33, 16)
    x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV)
    x = (x * torch.exp(4 * torch.randn(x.shape, generator=g, device=DEV))).bfloat16()
    w = torch.zeros((cfg.E, N, I // 2), dtype=torch.uint8, device=DEV)
    w[:, 1::3] = 0x73                                                # others beside them
    ws = torch.full((cfg.E, N, I // group), 0.75, dtype=torch.bfloat16, device=DEV)
    out, _ = _run(cfg, counts, x, w, ws, group)
    rows = sum(counts)
    zero = torch.ones(N, dtype=torch.bool, device=DEV)
    zero[1::3] = False
    assert (out[:rows, zero] == 0).all() and (out[:rows, ~zero] != 0).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_large_finite_rows_stay_finite(shape, group):
    """One code per group that is not 0: out is the sum over the groups of code * scale * x, two
    of them here, whose products are exact in fp32 and whose sum is too (a power of two and one
    that is 2^-4 of it)."""
    cfg, N = _config(shape)
    I = 2 * group
    counts = _counts(cfg.E, 20, 100, 33, 16)
    big = float(torch.finfo(torch.bfloat16).max)
    x = torch.full((cfg.expand_rows_capacity, I), big, dtype=torch.bfloat16, device=DEV)
    x[::2] = -big
    w = torch.zeros((cfg.E, N, I // 2), dtype=torch.uint8, device=DEV)
    code = torch.arange(N, device=DEV) % 16
    w[:, :, 3] = code.to(torch.uint8)                                # element 6 of the first group
    w[:, :, group // 2 + 5] = (code * 16).to(torch.uint8)            # element 11 of the second
    ws = torch.tensor([2.0 ** -8, 2.0 ** -12], device=DEV).bfloat16().expand(cfg.E, N, 2).contiguous()
    out, _ = _run(cfg, counts, x, w, ws, group)
    rows = sum(counts)
    value = torch.where(code > 7, code - 16, code).double()
    want = (x[:rows, :1].double() * value * (2.0 ** -8 + 2.0 ** -12)).float().bfloat16()
    assert torch.equal(out[:rows], want)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_a_row_does_not_depend_on_its_neighbours(shape, group):
    cfg, N = _config(shape)
    I = 5 * group
    g = torch.Generator(device=DEV).manual_seed(group + 1)
    w = torch.randint(0, 256, (cfg.E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = ((0.5 + torch.rand((cfg.E, N, I // group), generator=g, device=DEV)) /
          (4.6 * math.sqrt(I))).bfloat16()
    token = torch.randn((I,), generator=g, device=DEV).bfloat16()
    seen = None
    for n in (1, 16, 17, 32, 33, 64, 65, 96, 97, 128, 129, 300):
        x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV).bfloat16()
        x[[0, n - 1]] = token
        out, _ = _run(cfg, _counts(cfg.E, n, 7), x, w, ws, group)
        assert torch.equal(out[0], out[n - 1]), n
        if seen is not None:
            assert torch.equal(out[0], seen), n
        seen = out[0].clone()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_infinity_and_nan_stay_in_their_row(shape, group):
    cfg, N = _config(shape)
    I = 2 * group
    g = torch.Generator(device=DEV).manual_seed(group + 2)
    counts = _counts(cfg.E, 20, 70, 33, 16)
    rows = sum(counts)
    w = torch.randint(0, 256, (cfg.E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    w[:, :, 6] |= 0x10                                               # element 13 is not 0
    ws = torch.full((cfg.E, N, I // group), 0.25, dtype=torch.bfloat16, device=DEV)
    x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV).bfloat16()
    clean, ranges = _run(cfg, counts, x, w, ws, group)
    x[[0, 25, 89], 13] = math.inf
    x[[3, 40, 120], 13] = math.nan
    out, _ = _run(cfg, counts, x, w, ws, group)
    expert = torch.zeros(rows, dtype=torch.long, device=DEV)
    for e, (lo, hi) in enumerate(ranges):
        expert[lo:hi] = e
    sign = torch.where(w[expert, :, 6] >> 4 > 7, -1.0, 1.0)
    touched = torch.zeros(rows, dtype=torch.bool, device=DEV)
    touched[[0, 25, 89, 3, 40, 120]] = True
    assert torch.equal(out[[0, 25, 89]].float(), sign[[0, 25, 89]] * math.inf)
    assert torch.isnan(out[[3, 40, 120]]).all()
    assert torch.equal(out[:rows][~touched], clean[:rows][~touched])


RAGGED = [0, 1, 33, 64, 65, 97, 130, 161, 193, 225, 256, 257, 300, 511, 513, 769,
          31, 32, 0, 0, 16, 15, 2, 90, 224, 128, 129, 5, 48, 70, 0, 449]
FEW = [1, 0, 2, 33, 16, 17, 0, 5, 1, 1, 31, 32, 3, 70, 0, 8, 4, 12, 15, 64, 2, 2, 0, 9, 24, 25, 6, 7, 1, 0, 11, 130]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts,bs,N,swiglu,shape", [
    ([31, 33, 64, 65, 0, 7, 100, 129], 32, 160, False, "stream"), (FEW, 11, 770, False, "small"),
    (FEW, 11, 1666, True, "small"), (RAGGED, 102, 1541, False, "tiles"), (RAGGED, 102, 1602, True, "tiles"),
])
def test_sums_within_the_roundings_of_their_terms(counts, bs, N, swiglu, shape, group):
    """The bound of sums whose terms are code * scale * x, nothing besides."""
    W, K, I = 4, min(16, len(counts)), 9 * group
    cfg = cq.make_config(W, len(counts), bs, 1024, K)
    assert path("bf16", cfg, N, swiglu, "int4") == shape and sum(counts) <= cfg.expand_rows_capacity
    g = torch.Generator(device=DEV).manual_seed(group + N)
    rows, E = sum(counts), len(counts)
    erc, off, ranges = ref.pack_counts(counts, W)
    x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV).bfloat16()
    w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = ((0.5 + torch.rand((E, N, I // group), generator=g, device=DEV)) / (4.6 * math.sqrt(I))).bfloat16()
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_INT4, group_size=group,
                        activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))
    y, err = ref.product(x[:rows].double(), ref.w4_to_f64(w, ws, "int4", group), ranges, swiglu)
    ref.check(out, y, err, rows)
