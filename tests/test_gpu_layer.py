"""The experts' layer of a few tokens on the GPU against its plain 64-bit form (layer_ref)."""
import math

import pytest
import torch

import block_ref as blk
import combine_quant_amd as cq
import experts_ref as ref
import layer_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Case:
    """A layer with whole numbers: gates are 32 or more (so that silu changes nothing), up sums and
    weights small, so that h is exact in either token type and y is one rounding of a whole sum."""

    def __init__(self, W, BS, E, K, H, F, block=False, f16=False, zero=0, copy=0, mask_kind=0, seed=0, picks="any"):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.cfg = cq.make_config(W, E, BS, H, K, zero_expert_num=zero, copy_expert_num=copy, mask_kind=mask_kind,
                                  token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)
        token, T = cq.token_torch_dtype(self.cfg), W * BS
        rand = lambda lo, hi, *n: torch.randint(lo, hi + 1, n, generator=g, device=DEV)  # noqa: E731
        x = rand(-1, 1, T, H).float()
        x[:, 0] = 1.0
        self.x = x.to(token).view(W, BS, H)
        wt = torch.float8_e4m3fn if block else token
        up = torch.zeros((E, 2 * F, H), device=DEV)
        up[:, :F, 0] = 64.0 * rand(1, 2, E, F).float()
        at = rand(0, H - 1, E, F, 3)
        up[:, F:].scatter_(2, at, rand(-1, 1, E, F, 3).float())
        self.up = up.to(wt)
        self.down = rand(-2, 2, E, H, F).to(wt)
        self.ups = self.downs = None
        if block:
            power = lambda *n: 2.0 ** rand(-1, 1, *n).float()  # noqa: E731
            self.ups = power(E, 2 * blk.groups(F), blk.groups(H))
            self.downs = power(E, blk.groups(H), blk.groups(F))
        ids = E + zero + copy
        if picks == "any":                                   # the same expert twice is allowed
            self.ids = rand(0, ids - 1, W, BS, K).int()
        else:
            self.ids = torch.tensor(picks, device=DEV, dtype=torch.int32).view(W, BS, K)
        self.weight = rand(1, 2, W, BS, K).float()
        self.mask = None
        if mask_kind:
            self.mask = rand(0, 1, *((W, BS) if mask_kind == 1 else (W, BS, K))).to(torch.uint8)
        self.experts = cq.make_experts(F, cq.MOE_MM_SCALE_BLOCK if block else cq.MOE_MM_SCALE_NONE)
        self.shared = None

    def run(self, **kw):
        n = cq.moe_dc_experts_layer_workspace_bytes(self.cfg, self.experts)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)        # what it held must not matter
        y = cq.experts_layer(self.cfg, self.experts, self.x, self.ids, self.weight, self.up, self.down,
                             up_scales=self.ups, down_scales=self.downs, x_active_mask=self.mask,
                             shared_x=self.shared, workspace=ws, **kw)
        torch.cuda.synchronize()
        return y

    def plain(self):
        return layer_ref.layer(self.cfg, self.x.double().view(-1, self.cfg.hidden), self.ids, self.weight,
                               layer_ref.weights(self.up, self.ups, 2), layer_ref.weights(self.down, self.downs, 1),
                               self.mask, self.shared)

    def whole(self):
        """y; in 64 bits silu(t) for t >= 32 is still t (1 - 2^-46), in multiples of 2^-6 it is t."""
        y = torch.round(self.plain()[0] * 64) / 64
        assert y.abs().max() < 2 ** 24
        return y

    def check_exact(self):
        y = self.whole()
        out = self.run().view(y.shape)
        assert (out == y.float().to(out.dtype)).all(), int((out != y.float().to(out.dtype)).sum())


# W, BS, E, K: few and many tokens, experts shared by all tokens (up to 64 rows), more picks than ids
ROUTES = [(2, 1, 8, 2), (2, 1, 64, 8), (3, 1, 3, 1), (2, 4, 2, 4), (8, 2, 256, 16), (4, 5, 8, 3), (2, 16, 2, 5),
          (8, 4, 1024, 8), (3, 21, 3, 7), (2, 32, 4, 4), (32, 2, 32, 16)]


@pytest.mark.parametrize("block,f16", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("W,BS,E,K", ROUTES)
def test_routes(W, BS, E, K, block, f16):
    if E == 2 and K > 2:
        Case(W, BS, E, K, 1024, 144, block, f16, zero=1, copy=2, seed=K).check_exact()
    else:
        Case(W, BS, E, K, 1024, 48 if E > 100 else 144, block, f16, copy=max(0, K - E), seed=K).check_exact()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("H,F", [(1024, 16), (1040, 32), (1136, 528), (2064, 112), (7168, 128), (8192, 272),
                                 (1024, 2048), (1152, 4112)])
def test_sizes(H, F, block):
    Case(2, 3, 6, 3, H, F, block, seed=H + F).check_exact()


@pytest.mark.parametrize("H,F", [(1024, 8), (1032, 24), (1144, 520), (2056, 136)])
def test_sizes_of_token_weights(H, F):
    Case(2, 3, 6, 3, H, F, False, f16=F == 24, seed=H + F).check_exact()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("mask_kind", [1, 2])
@pytest.mark.parametrize("W,BS", [(2, 1), (2, 9), (4, 16)])
def test_masks_special_experts_and_shared_rows(W, BS, mask_kind, block):
    c = Case(W, BS, 8, 6, 1040, 160, block, zero=2, copy=3, mask_kind=mask_kind, seed=BS)
    c.shared = torch.randint(-9, 9, c.x.shape, device=DEV).to(c.x.dtype)
    c.check_exact()
    c.mask.zero_()
    assert (c.run() == c.shared).all()
    c.shared = None
    y = c.run()
    assert (y == 0).all() and not torch.signbit(y).any()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("H", [1024, 6144])
@pytest.mark.parametrize("E,K", [(1024, 16), (512, 2), (128, 16), (64, 16)])
def test_the_most_tokens(E, K, H, block):
    """64 tokens, with every number of rows that shares a sweep and the largest tables."""
    Case(2, 32, E, K, H, 16, block, seed=E).check_exact()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("H,F", [(1024, 32768), (8192, 4096)])
def test_largest_sizes(H, F, block):
    Case(2, 4, 2, 2, H, F, block, seed=1).check_exact()


def test_ids_out_of_range_count_as_inactive():
    c = Case(2, 3, 8, 4, 1024, 64, seed=3)
    c.ids[0, 1] = torch.tensor([-1, 8, 2 ** 31 - 1, -2 ** 31], device=DEV)
    c.ids[1, 0, 2] = 9
    y = c.whole()
    assert (c.run().view(y.shape) == y.float().to(c.x.dtype)).all()
    assert (c.run()[0, 1] == 0).all()


def test_one_expert_for_every_pick():
    c = Case(2, 32, 8, 5, 1024, 144, picks=[3] * 320)
    c.check_exact()
    Case(2, 32, 8, 5, 1024, 144, True, picks=[7] * 320).check_exact()


@pytest.mark.parametrize("W,BS,E,K,H,F", [(2, 1, 16, 4, 1024, 512), (2, 10, 8, 2, 2048, 1040), (2, 32, 8, 4, 1536, 256)])
@pytest.mark.parametrize("block,f16", [(False, False), (False, True), (True, False), (True, True)])
def test_values(W, BS, E, K, H, F, block, f16):
    c = Case(W, BS, E, K, H, F, block, f16, copy=1, seed=H)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
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
    c.shared = torch.randn(c.x.shape, generator=g, device=DEV).to(token)
    y, err = c.plain()
    out = c.run().view(y.shape)
    ref.check(out, y, err, len(y))
    # and what roundings do in the mean: h's and y's, a fraction of half a step each
    assert ((out.double() - y).norm() / y.norm()) < ref.HALF_STEP[token]
    for _ in range(3):
        assert (c.run().view(y.shape) == out).all()


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("BS", [2, 20])
def test_bad_weights_reach_their_tokens_only(block, bad, BS):
    c = Case(2, BS, 8, 3, 1040, 272, block, seed=11)
    c.ids[0, 0], c.ids[0, 1], c.ids[1, 0] = (torch.tensor(v) for v in ([2, 0, 1], [5, 3, 0], [6, 7, 0]))
    good = c.run().clone()
    if block:
        c.ups[5, 0, 1] = bad
        c.downs[2, 3, 0] = bad
    else:
        c.up[5, 7, 9] = bad
        c.down[2, 400, 3] = bad
    out = c.run()
    up_hit, down_hit = (c.ids == 5).any(2), (c.ids == 2).any(2)
    assert (out[~(up_hit | down_hit)] == good[~(up_hit | down_hit)]).all()
    cols = torch.zeros(1040, dtype=torch.bool, device=DEV)
    cols[384:512] = True if block else False
    cols[400] = True
    only = down_hit & ~up_hit
    assert only.any() and up_hit.any()
    assert (out[only][:, ~cols] == good[only][:, ~cols]).all()
    assert not torch.isfinite(out[only][:, 400]).any()
    assert not torch.isfinite(out[up_hit]).all(1).any()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_bad_tokens_stay_by_themselves(bad):
    c = Case(2, 6, 4, 3, 1024, 144, seed=13)
    good = c.run().clone()
    c.x[1, 2, 5] = bad
    out = c.run()
    keep = torch.ones((2, 6), dtype=torch.bool, device=DEV)
    keep[1, 2] = False
    assert (out[keep] == good[keep]).all()
