"""The layer of a few tokens is as near to 64 bits as one rounding of y: what lies before it, h among it,
is held in more bits.

Bound, root mean square relative to y: y's rounding alone gives r, at least 0.3 half steps (2^-9.8 bf16,
2^-12.8 fp16).  h's two parts leave 2^-17 (fp16: 2^-22, or 2^-25 absolute), SwiGLU 2^-17, the sums'
roundings in the mean below 2^-20 for these sizes: together below 2^-16, and sqrt(r^2 + 2^-32) <=
1.01 r.  With h rounded once the error would be 1.3 to 1.4 r.
"""
import math

import pytest
import torch

from test_gpu_layer import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"


# every number of rows that shares a sweep in the down product, 16 and 32 columns, runs that end early
@pytest.mark.parametrize("W,BS,E,K,H,F", [
    (2, 1, 16, 4, 1024, 512), (2, 2, 8, 2, 7168, 208), (2, 8, 8, 2, 2048, 1040), (2, 32, 64, 4, 1040, 272), (2, 32, 64, 4, 4608, 80),
    (2, 32, 64, 4, 6160, 144), (2, 32, 4, 4, 1536, 256), (2, 32, 4, 3, 6144, 336)])
@pytest.mark.parametrize("block,f16", [(False, False), (False, True), (True, False), (True, True)])
def test_one_rounding(W, BS, E, K, H, F, block, f16):
    c = Case(W, BS, E, K, H, F, block, f16, seed=H)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    token = c.x.dtype
    c.x = torch.randn(c.x.shape, generator=g, device=DEV).to(token)
    c.weight = torch.rand(c.weight.shape, generator=g, device=DEV)
    for name, n in (("up", H), ("down", F)):
        w = torch.randn(getattr(c, name).shape, generator=g, device=DEV)
        if block:
            setattr(c, name, (w * 60).to(torch.float8_e4m3fn))
            s = getattr(c, name + "s")
            setattr(c, name + "s", (0.3 + torch.rand(s.shape, generator=g, device=DEV)) / (60 * math.sqrt(n)))
        else:
            setattr(c, name, (w / math.sqrt(n)).to(token))
    y, _ = c.plain()
    out = c.run().view(y.shape)
    once = (y.to(token).double() - y).norm()
    assert (out.double() - y).norm() <= 1.01 * once, float((out.double() - y).norm() / once)


@pytest.mark.parametrize("block", [False, True])
def test_infinite_h_stays_infinite(block):
    """fp16: h past 65504 is infinite, and its rest is not a NaN that would hide it."""
    c = Case(2, 2, 4, 2, 1024, 48, block, f16=True, seed=1)
    c.up.zero_()
    c.up[:, :48, 0], c.up[:, 48:, 0] = 1.0, 1.0
    if block:
        c.ups.fill_(1.0)
        c.downs.fill_(1.0)
    c.down.zero_()
    c.down[:, ::2] = 1.0
    c.x[:, :, 0] = 300.0
    c.weight.fill_(0.5)
    out = c.run()
    # 300 * 300 = 90000; a zero weight meets an infinite h as NaN, as in any product
    assert torch.isposinf(out[..., ::2]).all() and out[..., 1::2].isnan().all()
