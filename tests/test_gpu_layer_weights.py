"""The picks' weights in the layer of a few tokens: they multiply fp32 sums, so that h is rounded as it
is, whatever the weight.  Sums are whole multiples of a power of two and exact, y is their one rounding."""
import pytest
import torch

import layer_ref
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu


# weight * h far below fp16's normal range, and far past its largest value (65504); h alone is 64 to 384
# times a whole number of at most 3, and y about 2^-11 and 2^10
@pytest.mark.parametrize("weight,down", [(3 * 2.0 ** -31, 2.0 ** 6), (2.0 ** 10, 2.0 ** -12)])
@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("W,BS,E,K", [(2, 1, 16, 2), (2, 8, 8, 3), (2, 32, 8, 5)])
def test_weights_do_not_change_the_rounding_of_h(W, BS, E, K, block, weight, down):
    c = Case(W, BS, E, K, 1024, 272, block, f16=True, seed=BS)
    c.weight *= weight
    if block:
        c.downs *= down
    else:
        c.down *= down
    unit = weight * down * 64 / 16                         # (scales of a block: 2^-1 to 2 each)
    y = torch.round(c.plain()[0] / unit)
    assert y.abs().max() < 2 ** 24
    y *= unit
    assert y.abs().max() < 60000 and y.abs().median() > 2.0 ** -14
    out = c.run().view(y.shape)
    want = y.float().half()
    assert (out == want).all(), int((out != want).sum())


@pytest.mark.parametrize("weight", [1e-3, 1e-5, 300.0])
def test_error_does_not_depend_on_the_weight(weight):
    """fp16, h near 1e-2: h's and y's roundings in the mean, less than half a step together (each is off
    by less than 0.6 of half a step, root mean square)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    c = Case(2, 8, 8, 3, 1024, 272, False, f16=True, seed=2)
    c.x = torch.randn(c.x.shape, generator=g, device="cuda").half()
    c.up = (torch.randn(c.up.shape, generator=g, device="cuda") * 0.1 / 32).half()
    c.down = (torch.randn(c.down.shape, generator=g, device="cuda") / weight).clamp(-60000, 60000).half()
    c.weight = weight * (0.5 + torch.rand(c.weight.shape, generator=g, device="cuda"))
    y, _ = c.plain()
    out = c.run().view(y.shape)
    assert (out.double() - y).norm() <= 2.0 ** -11 * y.norm()
