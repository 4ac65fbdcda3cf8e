"""SwiGLU of single products: gates over the whole range, where exp(-gate) passes the range of
binary32 and the up row brings the result back."""
import math

import pytest
import torch

import combine_quant_amd as cq
import experts_ref as ref
from experts_path import path

pytestmark = pytest.mark.gpu

DEV = "cuda"
GATES = [0.0, -0.0, 1.0, -1.0, 17.0, -17.0, 60.0, -60.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -96.0,
         -103.0, -104.0, -110.0, -120.0, -130.0, -150.0, -174.0, 88.0, 89.0, 200.0, -1000.0, 1000.0, 1e30, -1e30]
UPS = [1.0, -1.0, 2.0 ** -20, 2.0 ** 60, -2.0 ** 100, 2.0 ** 127, 0.0]


@pytest.mark.parametrize("w4", [None, "int4"])
@pytest.mark.parametrize("E,BS,want", [(4, 20, "stream"), (64, 20, "tiles"), (64, 512, "tiles")])
def test_gates_over_the_whole_range(E, BS, want, w4):
    """Row 0 of x picks out one weight each: the gate and up sums are the values themselves (int4:
    the scale carries them).  The result's error: 2^-17 of it for the exponential, the product and
    the division, half a step of bf16, and twice the least binary32 number where it is subnormal."""
    pairs = [(a, b) for a in GATES for b in UPS]
    n, I = len(pairs), 128
    cfg = cq.make_config(2, E, BS, 1024, 4)
    kind = path("bf16", cfg, 2 * n, True, w4)
    assert kind == ("small" if w4 and want == "tiles" and BS == 20 else want)
    v = torch.tensor([a for a, _ in pairs] + [b for _, b in pairs], device=DEV).bfloat16()
    erc, off, _ = ref.pack_counts([1, 0, 2] + [0] * (E - 3), 2)
    x = torch.zeros((cfg.expand_rows_capacity, I), dtype=torch.bfloat16, device=DEV)
    x[:3, 0] = 1.0
    if w4:
        w = torch.zeros((E, 2 * n, I // 2), dtype=torch.uint8, device=DEV)
        w[:, :, 0] = 1
        mm = cq.make_matmul(I, 2 * n, weight_dtype=cq.MOE_W4_INT4, group_size=128, activation=cq.MOE_ACT_SWIGLU)
        out = cq.grouped_matmul_w4(cfg, mm, x, w, v[None, :, None].expand(E, 2 * n, 1).contiguous(), erc.to(DEV),
                                   off.to(DEV))
    else:
        w = torch.zeros((E, 2 * n, I), dtype=torch.bfloat16, device=DEV)
        w[:, :, 0] = v
        mm = cq.make_matmul(I, 2 * n, activation=cq.MOE_ACT_SWIGLU)
        out = cq.grouped_matmul(cfg, mm, x, w, erc.to(DEV), off.to(DEV))
    a, b = v[:n].double(), v[n:].double()
    y = a * torch.exp(-torch.clamp(-a, min=0)) / (1 + torch.exp(-a.abs())) * b
    over = y.abs() > torch.finfo(torch.bfloat16).max * (1 + 2.0 ** -9)
    tol = y.abs() * (2.0 ** -17 + 2.0 ** -8) + 2.0 ** -133 + 2.0 ** -148
    for row in out[:3].double():
        assert torch.equal(row[over], y[over].sign() * math.inf)
        bad = (row - y).abs()[~over] > tol[~over]
        assert not bad.any(), [pairs[i] for i in (~over).nonzero().flatten()[bad].tolist()]


@pytest.mark.parametrize("E,BS,want", [(4, 20, "stream"), (64, 20, "tiles")])
def test_a_row_beside_rows_with_low_gates(E, BS, want):
    cfg = cq.make_config(2, E, BS, 1024, 4)
    N, I = 420, 128
    assert path("bf16", cfg, N, True) == want
    g = torch.Generator(device=DEV).manual_seed(2)
    erc, off, _ = ref.pack_counts([17, 0, 2] + [0] * (E - 3), 2)
    x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV).bfloat16()
    x[:, 0] = 0
    w = torch.randn((E, N, I), generator=g, device=DEV).bfloat16()
    w[:, :, 0] = -100.0
    mm = cq.make_matmul(I, N, activation=cq.MOE_ACT_SWIGLU)
    plain = cq.grouped_matmul(cfg, mm, x, w, erc.to(DEV), off.to(DEV)).clone()
    x[3, 0] = 1.0
    out = cq.grouped_matmul(cfg, mm, x, w, erc.to(DEV), off.to(DEV))
    keep = [r for r in range(19) if r != 3]
    assert torch.equal(out[keep], plain[keep]) and not torch.equal(out[3], plain[3])
