"""The RMS norm with residual and codes on the GPU against its plain 64-bit form.

Bounds: s has one rounding (2^-24, relative).  The sum of squares is formed in at most 32 steps of a
thread, 6 of a wave and 16 of a workgroup, each off by 2^-24 of the sum at most (its terms are of one
sign), the squares by 2^-24 and, through s, 2 * 2^-24; the root halves that (29 * 2^-24), and mean,
epsilon, root, reciprocal, two products and s itself add 7 * 2^-24: together below 2^-18.
"""
import math

import pytest
import torch

import combine_quant_amd as cq

pytestmark = pytest.mark.gpu

DEV = "cuda"
REL = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
TYPES = {"int8": (cq.MOE_DTYPE_INT8, torch.int8, 127.0), "e4m3": (cq.MOE_DTYPE_E4M3, torch.float8_e4m3fn, 448.0),
         "e5m2": (cq.MOE_DTYPE_E5M2, torch.float8_e5m2, 57344.0)}
CODE = {"int8": (0.0, 0.5), "e4m3": (2.0 ** -4, 2.0 ** -10), "e5m2": (2.0 ** -3, 2.0 ** -17)}   # half steps
EMAX = {"e4m3": 8, "e5m2": 15}


def _config(W, BS, H, mode, kind, fmt=cq.MOE_SCALE_FP32, f16=False):
    return cq.make_config(W, W, BS, H, 1, quant_mode=mode, out_dtype=TYPES[kind][0] if mode else 0,
                          scale_format=fmt, token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)


def _inputs(cfg, residual, seed, spread=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    shape, token = (cfg.ep_world_size, cfg.bs, cfg.hidden), cq.token_torch_dtype(cfg)
    x = torch.randn(shape, generator=g, device=DEV).to(token)
    r = None
    if residual:
        r = (torch.randn(shape, generator=g, device=DEV) * (1 + 7 * torch.rand(shape[:2] + (1,), generator=g, device=DEV)))
        r = (r * spread).to(token)
    return x, r, (torch.randn(shape[2:], generator=g, device=DEV)).to(token)


def _plain(x, r, gamma, eps):
    s = x.double() if r is None else x.double() + r.double()
    return s, s / torch.sqrt((s * s).mean(2, keepdim=True) + eps) * gamma.double()


def _near(out, want, rel):
    tol = rel * want.abs() + HALF[out.dtype] * want.abs() * (1 + rel) + TINY[out.dtype]
    assert ((out.double() - want).abs() <= tol).all()


def _split(v, width):
    H = v.shape[-1]
    return torch.nn.functional.pad(v, (0, -H % width)).view(*v.shape[:-1], -1, width)


def _check_codes(cfg, kind, codes, scales, y):
    mode, (half, least), top = cfg.quant_mode, CODE[kind], TYPES[kind][2]
    c = codes.view(TYPES[kind][1]).double()
    H, width = cfg.hidden, {2: cfg.hidden, 3: 128}.get(mode, 32)
    v, c = _split(y, width), _split(c, width)
    most = v.abs().amax(-1)
    if mode <= 3:
        s = scales.double().view(most.shape)
        assert ((s - most / top).abs() <= (REL + 2.0 ** -22) * most / top).all()
        tol = REL * v.abs() + (half + 2.0 ** -22) * v.abs() * (1 + REL) + least * s[..., None] * (1 + 2.0 ** -20)
        assert ((c * s[..., None] - v).abs() <= tol).all()
        return
    nb = most.shape[-1]
    if cfg.scale_format == cq.MOE_SCALE_E8M0:
        e = scales[..., :nb].double() - 127
    else:
        e = torch.log2(scales[..., :nb].double())
        if cfg.scale_format == cq.MOE_SCALE_FP32_RECIPROCAL:
            e = -e
    assert (scales[..., nb:] == 0).all() and scales.shape[-1] == nb + nb % 2

    def exponent(m):
        if mode == 4:
            return torch.where(m > 0, torch.floor(torch.log2(m.clamp_min(1e-300))) - EMAX[kind], -127.0).clamp_min(-127)
        return torch.ceil(torch.log2(m.clamp_min(1e-4) / top))
    lo, hi = exponent(most * (1 - REL)), exponent(most * (1 + REL))
    assert ((e == lo) | (e == hi)).all()
    scale = torch.exp2(e)[..., None]
    want = torch.maximum(torch.minimum(v, top * scale), -top * scale)
    assert ((c * scale - want).abs() <= REL * v.abs() + half * v.abs() * (1 + REL) + least * scale).all()


def _run(W, BS, H, mode, kind="e4m3", fmt=cq.MOE_SCALE_FP32, f16=False, residual=True, seed=0, eps=1e-6,
         misalign=False, spread=1.0):
    cfg = _config(W, BS, H, mode, kind, fmt, f16)
    x, r, gamma = _inputs(cfg, residual, seed, spread)
    if misalign:
        x = torch.cat([x.flatten()[:1], x.flatten()])[1:].view(x.shape)
        assert x.data_ptr() % 16
    out = cq.rms_norm(cfg, cq.make_norm(eps), x, gamma, residual=r)
    torch.cuda.synchronize()
    s, y = _plain(x, r, gamma, eps)
    if residual:
        _near(out["residual_out"], s, 2.0 ** -24)
    else:
        assert out["residual_out"] is None
    _near(out["y"], y, REL)
    if mode:
        _check_codes(cfg, kind, out["codes"], out["dynamic_scales"], y)


VARIANTS = [(0, "e4m3", 0), (2, "int8", 0), (2, "e4m3", 0), (2, "e5m2", 0), (3, "e4m3", 0), (3, "e5m2", 0),
            (4, "e4m3", 0), (4, "e5m2", 1), (4, "e4m3", 2), (5, "e4m3", 1), (5, "e5m2", 0)]


@pytest.mark.parametrize("H", [1024, 1032, 1144, 5128, 7168, 8192])
@pytest.mark.parametrize("mode,kind,fmt", VARIANTS)
def test_sizes(mode, kind, fmt, H):
    _run(3, 5, H, mode, kind, fmt, f16=H % 3 == 0, residual=H != 1144, seed=H + mode)


@pytest.mark.parametrize("mode,kind,fmt", VARIANTS)
def test_many_tokens(mode, kind, fmt):
    _run(4, 300, 2056, mode, kind, fmt, seed=mode)


@pytest.mark.parametrize("mode,kind,fmt", [VARIANTS[i] for i in (0, 1, 5, 7)])
def test_outputs_past_the_caches(mode, kind, fmt):
    _run(8, 300, 5256, mode, kind, fmt, seed=mode)


@pytest.mark.parametrize("H,misalign", [(1025, False), (1157, False), (8191, False), (2048, True)])
@pytest.mark.parametrize("mode,kind,fmt", VARIANTS)
def test_any_size_and_alignment(mode, kind, fmt, H, misalign):
    _run(2, 3, H, mode, kind, fmt, f16=mode == 3, residual=H != 1157, seed=H, misalign=misalign)


@pytest.mark.parametrize("H", [1024, 1027])
@pytest.mark.parametrize("eps", [1e-20, 1e-5, 10.0])
def test_epsilon_counts(eps, H):
    _run(2, 2, H, 3, eps=eps, spread=2.0 ** -12)


def test_the_largest_batch():
    """768 x 512 tokens of 8192: offsets past 32 bits."""
    cfg = _config(768, 512, 8192, 3, "e4m3")
    x = torch.zeros((768, 512, 8192), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    few = torch.randn((2, 512, 8192), generator=g, device=DEV).bfloat16()
    x[0], x[767] = few[0], few[1]
    gamma = torch.randn((8192,), generator=g, device=DEV).bfloat16()
    out = cq.rms_norm(cfg, cq.make_norm(), x, gamma)
    torch.cuda.synchronize()
    _, y = _plain(few, None, gamma, 1e-6)
    _near(out["y"][[0, 767]], y, REL)
    _check_codes(cfg, "e4m3", out["codes"][[0, 767]], out["dynamic_scales"][[0, 767]], y)
    assert (out["y"][1:767] == 0).all() and (out["dynamic_scales"][1:767] == 0).all()


def test_repeats_its_bytes():
    cfg = _config(3, 500, 1152, 3, "e4m3")
    x, r, gamma = _inputs(cfg, True, 1)
    a = cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r)
    b = cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r)
    for k in a:
        assert (a[k] == b[k]).all()


@pytest.mark.parametrize("H", [1024, 1031])
def test_in_place(H):
    cfg = _config(2, 3, H, 2, "int8")
    x, r, gamma = _inputs(cfg, True, 2)
    want = cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r)
    out = dict(want, residual_out=r, y=x, codes=torch.empty_like(want["codes"]),
               dynamic_scales=torch.empty_like(want["dynamic_scales"]))
    cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r, out=out)
    for k in want:
        assert (out[k] == want[k]).all()


@pytest.mark.parametrize("H", [1024, 1031])
def test_outputs_left_out(H):
    cfg = _config(2, 3, H, 3, "e4m3")
    x, r, gamma = _inputs(cfg, True, 3)
    want = cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r)
    out = {k: torch.empty_like(want[k]) for k in ("codes", "dynamic_scales")}
    cq.rms_norm(cfg, cq.make_norm(), x, gamma, residual=r, out=out)
    for k in out:
        assert (out[k] == want[k]).all()


@pytest.mark.parametrize("H", [1024, 1031])
@pytest.mark.parametrize("mode,kind,fmt", VARIANTS[1:])
def test_zero_and_bad_tokens(mode, kind, fmt, H):
    cfg = _config(2, 4, H, mode, kind, fmt)
    x, _, gamma = _inputs(cfg, False, 4)
    good = cq.rms_norm(cfg, cq.make_norm(), x, gamma)
    x[0, 1] = 0.0
    x[0, 3, 5] = math.nan
    x[1, 2, H - 1] = math.inf
    out = cq.rms_norm(cfg, cq.make_norm(), x, gamma)
    torch.cuda.synchronize()
    for w, b in ((0, 0), (0, 2), (1, 0), (1, 1), (1, 3)):
        for k in ("y", "codes", "dynamic_scales"):
            assert (out[k][w, b] == good[k][w, b]).all()
    assert (out["y"][0, 1] == 0).all() and (out["codes"][0, 1].view(torch.uint8) & 0x7F == 0).all()
    assert out["y"][0, 3].isnan().all() and out["y"][1, 2, H - 1].isnan() and (out["y"][1, 2, :H - 1] == 0).all()
    s, nb = out["dynamic_scales"], (H + 31) // 32
    bad = (lambda t: t == 255) if fmt == cq.MOE_SCALE_E8M0 else torch.isnan
    if mode == 2:
        assert s[0, 1] == 0 and s[0, 3].isnan() and s[1, 2].isnan()
    elif mode == 3:
        assert (s[0, 1] == 0).all() and s[0, 3].isnan().all() and s[1, 2, -1].isnan() and (s[1, 2, :-1] == 0).all()
    else:
        assert bad(s[0, 3, :nb]).all() and bad(s[1, 2, nb - 1]) and not bad(s[1, 2, :nb - 1]).any()
    assert (out["codes"][0, 3] == 0).all()


def test_codes_equal_dispatch_of_the_same_values():
    """A norm that changes nothing (every token of one magnitude, gamma 1) codes a token as
    dispatch does."""
    W, BS, H = 2, 4, 1152
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    # +-1 everywhere: mean square 1, and 1 + epsilon rounds to 1
    x = (torch.randint(0, 2, (W, BS, H), generator=g, device=DEV) * 2 - 1).to(torch.bfloat16)
    gamma = torch.randn((H,), generator=g, device=DEV).to(torch.bfloat16)
    for mode, kind, fmt in VARIANTS[1:]:
        cfg = _config(W, BS, H, mode, kind, fmt)
        n = cq.rms_norm(cfg, cq.make_norm(1e-9), x, gamma)
        assert (n["y"] == x * gamma).all()
        ids = torch.arange(W, device=DEV, dtype=torch.int32).view(W, 1, 1).expand(W, BS, 1).contiguous()
        d = cq.dispatch(cfg, n["y"], ids)
        torch.cuda.synchronize()
        assert (d["expand_x"].view(W, BS, H).view(torch.uint8) == n["codes"].view(torch.uint8)).all()
        assert (d["dynamic_scales"].view(W * BS, -1) == n["dynamic_scales"].view(W * BS, -1)).all()
