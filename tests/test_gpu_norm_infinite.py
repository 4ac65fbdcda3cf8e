"""Norms whose y leaves the range of fp32 although the token is finite: an infinite gamma, and a gamma
that is nearly.  The scale of what holds such a value is NaN, whatever the mode; the rest is as it was."""
import math

import pytest
import torch

import combine_quant_amd as cq
from test_gpu_norm import VARIANTS, _config, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("H", [1024, 1031])
@pytest.mark.parametrize("mode,kind,fmt", VARIANTS[1:])
def test_infinite_values(mode, kind, fmt, H, bad):
    cfg = _config(2, 3, H, mode, kind, fmt)
    x, _, gamma = _inputs(cfg, False, 6)
    x[:, :, 300] = 20.0 + x[:, :, 300].abs()                # times 3e38 past the range
    good = cq.rms_norm(cfg, cq.make_norm(), x, gamma)
    gamma[300] = bad
    out = cq.rms_norm(cfg, cq.make_norm(), x, gamma)
    torch.cuda.synchronize()
    assert torch.isinf(out["y"][:, :, 300]).all()
    width = {2: H, 3: 128}.get(mode, 32)
    n = -(-H // width)
    s, gs = (t["dynamic_scales"].view(2, 3, -1) for t in (out, good))
    hit = torch.zeros(s.shape[2], dtype=torch.bool, device=s.device)
    hit[300 // width] = True
    nan = (lambda t: t == 255) if fmt == cq.MOE_SCALE_E8M0 else torch.isnan
    assert nan(s[:, :, hit]).all(), s[:, :, hit]
    assert not nan(s[:, :, ~hit]).any() and (s[:, :, ~hit] == gs[:, :, ~hit]).all()
    keep = ~hit[:n].repeat_interleave(width)[:H]
    assert (out["codes"].view(torch.uint8)[..., keep] == good["codes"].view(torch.uint8)[..., keep]).all()
    if mode <= 3:                                           # as in any group with a NaN
        assert (out["codes"].view(torch.uint8)[..., ~keep] & 0x7F == 0).all()
