"""The experts' products on values whose sums are exact: small whole numbers with scales that are
powers of two, so that every partial sum is a whole multiple of one power of two, of less than 2^24
of them, and no rounding takes place before the result's own.  A lost, doubled or misplaced element
shows as another value, whatever the inner size.

SwiGLU is exact too where every gate is at least 18: exp(-18) < 2^-25, so 1 + exp(-gate) rounds to
1, the gate is its own silu, and gate * up is one fp32 product.

(The fp8 matrix instructions cut products at 2^-13 of the power of two of the largest of eight: the
products here are whole multiples of 1/4 and at most 36, so nothing lies below 2^-13 * 2^5.)
"""
import math

import pytest
import torch

import combine_quant_amd as cq
import experts_ref as ref
from experts_path import path

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = ("bf16", "f16", "int8", "e4m3", "e5m2", "mx_e4m3", "mx_e5m2")
CODES = {"bf16": torch.bfloat16, "f16": torch.float16, "int8": torch.int8,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SCALES = torch.tensor([126, 127, 128], dtype=torch.uint8)             # 1/2, 1, 2
W4 = [("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _config(W, counts, f16=False, bs=None):
    K = min(16, len(counts))
    bs = bs or max(1, -(-sum(counts) // (W * K)))
    assert bs <= 512 and sum(counts) <= W * bs * K
    return cq.make_config(W, len(counts), bs, 1024, K,
                          token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)


def _whole(shape, lo, hi, g):
    return torch.randint(lo, hi + 1, shape, generator=g, device=DEV).float()


def _at_the_end(t):
    """The same tensor at the end of what a buffer holds of it, bytes of 255 behind."""
    n = t.numel() * t.element_size()
    buf = torch.full((n + 64,), 255, dtype=torch.uint8, device=DEV)
    buf[:n] = t.contiguous().view(torch.uint8).flatten()
    return buf[:n].view(t.dtype).view(t.shape)


def _scales(shape, g):
    return SCALES.to(DEV)[torch.randint(0, 3, shape, generator=g, device=DEV)]


def _desc(kind, I, N, swiglu):
    x_dtype = {"int8": cq.MOE_DTYPE_INT8, "e4m3": cq.MOE_DTYPE_E4M3, "e5m2": cq.MOE_DTYPE_E5M2}.get(
        kind.split("_")[-1], 0)
    scaling = (cq.MOE_MM_SCALE_MX if kind.startswith("mx") else
               cq.MOE_MM_SCALE_ROW if x_dtype else cq.MOE_MM_SCALE_NONE)
    return cq.make_matmul(I, N, x_dtype=x_dtype, scaling=scaling,
                          activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)


def _want(s, swiglu, dt):
    """fp64 sums (exact) -> the result: fp32, with SwiGLU one fp32 product, one rounding."""
    s = s.float()
    if swiglu:
        half = s.shape[1] // 2
        assert (s[:, :half] >= 18).all()
        s = s[:, :half] * s[:, half:]
    return s.to(dt)


def _compare(out, x, w, ranges, swiglu, filler):
    """x [R][I], w [E][N][I] as fp64 values."""
    rows = ranges[-1][1]
    for e, (lo, hi) in enumerate(ranges):
        if lo < hi:
            s = x[lo:hi] @ w[e].t()
            assert float(s.abs().max()) < 2 ** 20
            got, want = out[lo:hi], _want(s, swiglu, out.dtype)
            bad = got != want
            assert not bad.any(), (e, hi - lo, int(bad.sum()), bad.nonzero()[0].tolist())
    assert (out[rows:] == filler).all()


def _run(kind, W, counts, I, N, swiglu, want_path, bs=None, seed=0):
    g = _gen(seed)
    f16 = kind == "f16"
    cfg = _config(W, counts, f16, bs)
    assert path(kind, cfg, N, swiglu) == want_path
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    erc, off, ranges = ref.pack_counts(counts, W)
    elem = kind.split("_")[-1]
    x = _whole((cap, I), 1 if swiglu else -3, 3, g).to(CODES[elem])
    w = _whole((E, N, I), -3, 3, g)
    if swiglu:
        w[:, :N // 2] = w[:, :N // 2].abs() + 1                      # gates are positive
    w = w.to(CODES["e4m3"] if elem == "e5m2" else CODES[elem])
    xs = ws = None
    if kind.startswith("mx"):
        xs, ws = _scales((cap, I // 32), g), _scales((E, N, I // 32), g)
    elif elem not in ("bf16", "f16"):
        xs, ws = ref.power(_scales((cap,), g)).float(), ref.power(_scales((E, N), g)).float()
    vx, vw = ref.codes_to_f64(x, xs), ref.codes_to_f64(w, ws)
    if rows < cap:                              # what lies behind the last row must not matter
        x.view(torch.uint8)[rows:] = 0x7F
    args = [None if t is None else _at_the_end(t) for t in (x, w, xs, ws)]
    out = torch.full((cap, N // 2 if swiglu else N), 7.25, device=DEV,
                     dtype=torch.float16 if f16 else torch.bfloat16)
    cq.grouped_matmul(cfg, _desc(kind, I, N, swiglu), args[0], args[1], erc.to(DEV), off.to(DEV),
                      x_scales=args[2], weight_scales=args[3], out=out)
    torch.cuda.synchronize()
    _compare(out, vx[:rows], vw, ranges, swiglu, 7.25)


def _run_w4(token, weight, group, W, counts, I, N, swiglu, want_path, bs=None, seed=0):
    g = _gen(seed)
    f16 = token == "f16"
    dt = torch.float16 if f16 else torch.bfloat16
    cfg = _config(W, counts, f16, bs)
    assert path(token, cfg, N, swiglu, weight) == want_path
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    erc, off, ranges = ref.pack_counts(counts, W)
    x = _whole((cap, I), 1 if swiglu else -3, 3, g).to(dt)
    w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    if swiglu:
        w[:, :N // 2] = (w[:, :N // 2] & 0x77) | 0x22                # gates are positive
    ws = _scales((E, N, I // group), g)
    if weight == "int4":
        ws = ref.power(ws).to(dt)
    values = ref.w4_to_f64(w, ws, weight, group)
    x[rows:] = float("nan")
    out = torch.full((cap, N // 2 if swiglu else N), 7.25, device=DEV, dtype=dt)
    mm = cq.make_matmul(I, N, weight_dtype=W4_DTYPE[weight], group_size=group,
                        activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)
    cq.grouped_matmul_w4(cfg, mm, _at_the_end(x), _at_the_end(w), _at_the_end(ws), erc.to(DEV),
                         off.to(DEV), out=out)
    torch.cuda.synchronize()
    _compare(out, x[:rows].double(), values, ranges, swiglu, 7.25)


W4_DTYPE = {"int4": cq.MOE_W4_INT4, "e2m1": cq.MOE_W4_E2M1}


# -- MX scales where a row's last 16 bytes of them are not whole ------------------------------------

@pytest.mark.parametrize("kind", ["mx_e4m3", "mx_e5m2"])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 9, 16, 18])
@pytest.mark.parametrize("counts,N,swiglu,want", [
    ([33, 0, 64, 15], 100, False, "stream"),
    ([33, 0, 64, 15, 192, 1, 256, 16] * 4, 514, False, "tiles"),
    ([33, 0, 64, 15, 192, 1, 256, 16] * 4, 772, True, "tiles"),
])
def test_mx_scales_of_every_number_of_steps(kind, steps, counts, N, swiglu, want):
    """The last row's scales end where the tensor does."""
    _run(kind, 4, counts, 128 * steps, N, swiglu, want, seed=steps)


# -- products of every kind through each kernel ----------------------------------------------------

def _spread(E, live, rows):
    """`rows` rows on the experts `live`, of differing counts, none elsewhere."""
    counts = [0] * E
    share = [1 + (7 * i) % 13 for i in range(len(live))]
    for e, s in zip(live, share):
        counts[e] = max(1, rows * s // sum(share))
    return counts


def _many(E):
    """Counts on most experts, the first and the last few of them empty."""
    return [0 if e < 2 or e > E - 3 or e % 7 == 3 else (e * 5) % 39 + (e % 31 == 8) * 250 for e in range(E)]


# (E, W, counts): more experts than one wave counts by itself, and the most that one does; experts
# with rows on both sides of where one wave's share of the table ends (128 experts in a workgroup
# of eight waves, 256 in one of four)
EXPERTS = [(128, 4, _many(128)), (129, 3, _many(129)), (256, 8, _many(256)), (1024, 8, _many(1024)),
           (256, 8, _spread(256, [126, 127, 128, 129], 700)),
           (1024, 8, _spread(1024, [0, 255, 256, 257, 511, 512, 1023], 900)),
           (1024, 4, _spread(1024, [1023], 5)), (130, 2, _spread(130, [0, 129], 330))]
IDS = [f"{E}x{sum(c)}" for E, _, c in EXPERTS]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("E,W,counts", EXPERTS, ids=IDS)
def test_many_experts(kind, E, W, counts):
    step = 128 if kind.startswith("mx") else 144
    least = 56 // min(E, W * 16 * max(1, -(-sum(counts) // (W * 16)))) + 1
    _run(kind, W, counts, step, max(200, 256 * least - 3), False, "tiles", seed=E)


@pytest.mark.parametrize("kind", ["bf16", "int8", "e4m3", "mx_e5m2"])
@pytest.mark.parametrize("E,W,counts", EXPERTS[1:4], ids=IDS[1:4])
def test_many_experts_with_swiglu(kind, E, W, counts):
    _run(kind, W, counts, 256, 386, True, "tiles", seed=E)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("E,W,counts", EXPERTS, ids=IDS)
def test_4bit_many_experts(token, weight, group, E, W, counts):
    """The small tiles (the config's rows are few), and the large ones (they are many)."""
    cfg = _config(W, counts)
    rows = W * cfg.bs * cfg.topk
    active = min(E, rows)
    least = 144 // active + 1
    _run_w4(token, weight, group, W, counts, 3 * group, max(200, 128 * least - 3), False, "small",
            bs=cfg.bs if rows <= 32 * active else None, seed=E)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("E,W,counts", EXPERTS[:6], ids=IDS[:6])
@pytest.mark.parametrize("swiglu", [False, True])
def test_4bit_many_experts_large_tiles(token, weight, group, E, W, counts, swiglu):
    _run_w4(token, weight, group, W, counts, 2 * group, 260, swiglu, "tiles", bs=33 * E // (W * 16) + 1, seed=E)


# one expert with more than eight tiles of rows (a second band), others with rows around whole tiles
LONG = [700, 0, 257, 512, 2500, 1025, 385, 255]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_rows_through_tiles(kind, swiglu):
    step = 128 if kind.startswith("mx") else 48
    _run(kind, 2, LONG, step * 7, 520, swiglu, "tiles", seed=3)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("swiglu", [False, True])
def test_4bit_many_rows_through_tiles(token, weight, group, swiglu):
    _run_w4(token, weight, group, 2, LONG, group * 7, 520, swiglu, "tiles", seed=3)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("counts,N,swiglu,want", [
    ([5, 0, 90, 21], 131, False, "stream"), ([5, 0, 90, 21], 130, True, "stream"),
    ([5, 0, 90, 300, 16, 1, 17, 129] * 2, 1100, False, "tiles"), ([5, 0, 90, 300] * 4, 1100, True, "tiles"),
])
@pytest.mark.parametrize("I", [128, 640, 5248])
def test_long_and_short_rows(kind, counts, N, swiglu, want, I):
    _run(kind, 2, counts, I, N, swiglu, want, seed=I)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("counts,N,swiglu,want", [
    ([5, 0, 90, 21], 131, False, "stream"), ([5, 0, 90, 21], 130, True, "stream"),
    ([5, 0, 9, 33, 16, 1, 17, 70] * 4, 770, False, "small"), ([5, 0, 90, 300] * 8, 770, True, "tiles"),
])
@pytest.mark.parametrize("groups", [2, 5, 41])
def test_4bit_long_and_short_rows(token, weight, group, counts, N, swiglu, want, groups):
    _run_w4(token, weight, group, 2, counts, groups * group, N, swiglu, want, seed=groups)


@pytest.mark.parametrize("counts,N,want", [([3, 0], 33, "stream"), ([3, 0, 40, 1] * 14, 17, "tiles")])
def test_largest_int8_sums(counts, N, want):
    """65536 products of -128 and -128: 2^30, exact in 32 bits."""
    W, I, E = 2, 65536, len(counts)
    cfg = _config(W, counts)
    assert path("int8", cfg, N, False) == want
    erc, off, _ = ref.pack_counts(counts, W)
    x = torch.full((cfg.expand_rows_capacity, I), -128, dtype=torch.int8, device=DEV)
    w = torch.full((E, N, I), -128, dtype=torch.int8, device=DEV)
    x[::2, 77] = -127                                                # 2^30 - 128
    ws = torch.full((E, N), 2.0 ** -6, device=DEV)
    out = cq.grouped_matmul(cfg, _desc("int8", I, N, False), x, w, erc.to(DEV), off.to(DEV), weight_scales=ws)
    rows = sum(counts)
    want = torch.full((rows, 1), 2.0 ** 30, dtype=torch.float64, device=DEV)
    want[::2] -= 128
    assert torch.equal(out[:rows], (want * 2.0 ** -6).float().bfloat16().expand(rows, N))


@pytest.mark.parametrize("counts,N,want", [([5, 0, 90, 21], 131, "stream"),
                                          ([5, 0, 90, 300, 16, 1, 17, 129] * 2, 1100, "tiles")])
def test_int8_to_the_last_bit(counts, N, want):
    """Any codes and scales: the sum rounded to fp32, times the weight row's scale, times the
    row's, each rounded, and the result rounded to bf16."""
    W, I, E = 2, 1392, len(counts)
    g = _gen(8)
    cfg = _config(W, counts)
    assert path("int8", cfg, N, False) == want
    erc, off, ranges = ref.pack_counts(counts, W)
    rows = sum(counts)
    x = _whole((cfg.expand_rows_capacity, I), -128, 127, g).to(torch.int8)
    w = _whole((E, N, I), -128, 127, g).to(torch.int8)
    xs = 0.001 + torch.rand((cfg.expand_rows_capacity,), generator=g, device=DEV)
    ws = 0.001 + torch.rand((E, N), generator=g, device=DEV)
    out = cq.grouped_matmul(cfg, _desc("int8", I, N, False), x, w, erc.to(DEV), off.to(DEV), x_scales=xs,
                            weight_scales=ws)
    for e, (lo, hi) in enumerate(ranges):
        s = (x[lo:hi].double() @ w[e].double().t()).float()
        assert torch.equal(out[lo:hi], (s * ws[e] * xs[lo:hi, None]).bfloat16()), e


# -- one row among others ------------------------------------------------------------------------

PATHS = {"stream": (4, 80, 70), "tiles": (32, 256, 770)}               # experts, tokens a rank, N


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("want", PATHS)
def test_a_row_does_not_depend_on_its_neighbours(kind, want):
    E, BS, N = PATHS[want]
    I = 640
    cfg = cq.make_config(2, E, BS, 1024, 4, token_dtype=int(kind == "f16"))
    assert path(kind, cfg, N, False) == want
    g = _gen(4)
    elem = kind.split("_")[-1]
    cap = cfg.expand_rows_capacity

    def codes(shape, weights=False):
        v = torch.randn(shape, generator=g, device=DEV)
        if elem == "int8":
            return (v * 40).round().clamp(-127, 127).to(torch.int8)
        return v.to(CODES["e4m3" if weights and elem == "e5m2" else elem])

    w = codes((E, N, I), True)
    ws = _scales((E, N, I // 32), g) if kind.startswith("mx") else (
        0.1 + torch.rand((E, N), generator=g, device=DEV) if elem not in ("bf16", "f16") else None)
    token, seen = codes((I,)), None
    for n in (1, 15, 16, 17, 32, 33, 48, 64, 65, 100, 129, 192, 193, 256, 257, 300):
        x = codes((cap, I))
        x[[0, n - 1]] = token
        xs = None
        if kind.startswith("mx"):
            xs = _scales((cap, I // 32), g)
            xs[[0, n - 1]] = 127
        elif ws is not None:
            xs = 0.1 + torch.rand((cap,), generator=g, device=DEV)
            xs[[0, n - 1]] = 0.5
        erc, off, _ = ref.pack_counts([n, 7] + [0] * (E - 2), 2)
        out = cq.grouped_matmul(cfg, _desc(kind, I, N, False), x, w, erc.to(DEV), off.to(DEV), x_scales=xs,
                                weight_scales=ws)
        assert torch.equal(out[0], out[n - 1]), n
        assert seen is None or torch.equal(out[0], seen), n
        seen = out[0].clone()


# -- NaN and infinity ------------------------------------------------------------------------------

NONFINITE = [(k, v, p) for k, v in
             [("bf16", 0x7F80), ("bf16", 0xFF80), ("bf16", 0x7FC0), ("f16", 0x7C00), ("f16", 0x7E00), ("e4m3", 0x7F),
              ("e5m2", 0x7C), ("e5m2", 0xFC), ("e5m2", 0x7F), ("mx_e4m3", 0x7F), ("mx_e5m2", 0x7C), ("mx_e5m2", 0x7E)]
             for p in ("stream", "tiles")]


def _inf_or_nan(kind, bits):
    """+1 or -1 for an infinity of that sign, None for NaN."""
    if bits in {"bf16": (0x7F80, 0xFF80), "f16": (0x7C00,), "e4m3": (), "e5m2": (0x7C, 0xFC)}[kind.split("_")[-1]]:
        return -1.0 if bits >> (15 if kind in ("bf16", "f16") else 7) else 1.0
    return None


def _setup(kind, want, I, extra=0):
    E, BS, N = PATHS[want]
    cfg = cq.make_config(2, E, BS, 1024, 4, token_dtype=int(kind == "f16"))
    assert path(kind, cfg, N, False) == want
    g = _gen(6)
    elem = kind.split("_")[-1]
    x = _whole((cfg.expand_rows_capacity, I), 1, 3, g).to(CODES[elem])
    w = _whole((E, N, I), 1, 3, g)
    w = (w * _whole((E, N, 1), 0, 1, g).mul(2).sub(1)).to(CODES["e4m3" if elem == "e5m2" else elem])
    xs = ws = None
    if kind.startswith("mx"):
        xs, ws = _scales((x.shape[0], I // 32), g), _scales((E, N, I // 32), g)
    elif elem not in ("bf16", "f16"):
        xs, ws = torch.ones((x.shape[0],), device=DEV), torch.ones((E, N), device=DEV)
    counts = [20, 70, 0, 193] + [0] * (E - 4)
    erc, off, ranges = ref.pack_counts(counts, 2)
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to(DEV)

    def run():
        return cq.grouped_matmul(cfg, _desc(kind, I, N, False), x, w, erc.to(DEV), off.to(DEV), x_scales=xs,
                                 weight_scales=ws)[:sum(counts)].clone()
    return x, w, xs, ws, expert, run


def _bits(t):
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16)


def _signed(bits, t):
    return bits - 65536 if t.element_size() == 2 and bits > 0x7FFF else bits


@pytest.mark.parametrize("kind,bits,want", NONFINITE)
def test_nonfinite_rows(kind, bits, want):
    x, w, _, _, expert, run = _setup(kind, want, 384)
    clean = run()
    bad = [0, 19, 25, 90, 282]
    _bits(x)[bad, 301] = _signed(bits, x)
    out = run()
    good = torch.ones(len(clean), dtype=torch.bool, device=DEV)
    good[bad] = False
    assert torch.equal(out[good], clean[good]) and torch.isfinite(clean.float()).all()
    sign = _inf_or_nan(kind, bits)
    if sign is None:
        assert torch.isnan(out[bad].float()).all()
    else:
        assert torch.equal(out[bad].float(), w[expert[bad], :, 301].float().sign() * sign * math.inf)


@pytest.mark.parametrize("kind,bits,want", [c for c in NONFINITE if "e5m2" not in c[0]])
def test_nonfinite_weight_rows(kind, bits, want):
    x, w, _, _, expert, run = _setup(kind, want, 384)
    clean = run()
    bad = [0, 15, 17, 31, 40, 69]
    _bits(w)[:, bad, 130] = _signed(bits, w)
    out = run()
    good = torch.ones(clean.shape[1], dtype=torch.bool, device=DEV)
    good[bad] = False
    assert torch.equal(out[:, good], clean[:, good])
    sign = _inf_or_nan(kind, bits)                                   # (every x is positive)
    assert torch.isnan(out[:, bad].float()).all() if sign is None else (out[:, bad].float() == sign * math.inf).all()


@pytest.mark.parametrize("kind", ["mx_e4m3", "mx_e5m2"])
@pytest.mark.parametrize("want", PATHS)
@pytest.mark.parametrize("I", [128, 384, 640, 2048])
def test_nan_scales(kind, want, I):
    """A block's scale that is NaN, the last or the first of its row, stays in that row."""
    x, w, xs, ws, expert, run = _setup(kind, want, I)
    clean = run()
    xs[[3, 88], -1] = 255
    xs[[7, 89, 282], 0] = 255
    ws[:, [2, 33], -1] = 255
    ws[:, [16, 69], 0] = 255
    out = run()
    row = torch.ones(len(clean), dtype=torch.bool, device=DEV)
    row[[3, 88, 7, 89, 282]] = False
    col = torch.ones(clean.shape[1], dtype=torch.bool, device=DEV)
    col[[2, 33, 16, 69]] = False
    assert torch.equal(out[row][:, col], clean[row][:, col])
    assert torch.isnan(out[~row].float()).all() and torch.isnan(out[:, ~col].float()).all()


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("counts,N,want", [([5, 0, 18, 2], 33, "stream"), ([5, 0, 18, 33] * 8, 770, "small"),
                                          ([5, 0, 90, 129] * 8, 770, "tiles")])
@pytest.mark.parametrize("groups", [1, 3, 4, 5, 8, 9])
def test_4bit_infinite_first_and_last_scales(token, group, counts, N, want, groups):
    """Weight rows in turn: all scales 1; the last infinite; the first infinite.  A row of ones next
    to them keeps its sum, whichever part of a chunk its end falls in."""
    dt = torch.float16 if token == "f16" else torch.bfloat16
    W, E, I = 2, len(counts), group * groups
    cfg = _config(W, counts, token == "f16")
    assert path(token, cfg, N, False, "int4") == want
    erc, off, _ = ref.pack_counts(counts, W)
    x = torch.ones((cfg.expand_rows_capacity, I), dtype=dt, device=DEV)
    w = torch.full((E, N, I // 2), 0x11, dtype=torch.uint8, device=DEV)
    w[:, 2::3] = 0xFF                                                # -1
    ws = torch.ones((E, N, groups), dtype=dt, device=DEV)
    ws[:, 1::3, -1] = math.inf
    ws[:, 2::3, 0] = math.inf
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_INT4, group_size=group)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, _at_the_end(ws), erc.to(DEV), off.to(DEV))[:sum(counts)].float()
    assert (out[:, ::3] == torch.tensor(float(I), device=DEV).to(dt).float()).all()
    assert (out[:, 1::3] == math.inf).all() and (out[:, 2::3] == -math.inf).all()


@pytest.mark.parametrize("token,bits", [("bf16", 0x7F80), ("bf16", 0x7FC0), ("f16", 0x7C00), ("f16", 0x7E00)])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("counts,N,want", [([5, 0, 18, 2], 33, "stream"), ([5, 0, 18, 33] * 8, 770, "small"),
                                          ([5, 0, 90, 129] * 8, 770, "tiles")])
def test_4bit_nonfinite_rows(token, bits, weight, group, counts, N, want):
    dt = torch.float16 if token == "f16" else torch.bfloat16
    W, E, I = 2, len(counts), 3 * group
    g = _gen(group)
    cfg = _config(W, counts, token == "f16")
    assert path(token, cfg, N, False, weight) == want
    erc, off, _ = ref.pack_counts(counts, W)
    rows = sum(counts)
    expert = torch.repeat_interleave(torch.arange(E), torch.tensor(counts)).to(DEV)
    x = _whole((cfg.expand_rows_capacity, I), -3, 3, g).to(dt)
    w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    w[:, :, 20] |= 0x01                                              # element 40 is not 0
    ws = _scales((E, N, I // group), g)
    if weight == "int4":
        ws = ref.power(ws).to(dt)
    mm = cq.make_matmul(I, N, weight_dtype=W4_DTYPE[weight], group_size=group)
    clean = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))[:rows].clone()
    bad = [0, 4, 7, rows - 1]
    x.view(torch.int16)[bad, 40] = bits
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))[:rows]
    good = torch.ones(rows, dtype=torch.bool, device=DEV)
    good[bad] = False
    assert torch.equal(out[good], clean[good])
    if _inf_or_nan(token, bits) is None:
        assert torch.isnan(out[bad].float()).all()
    else:
        sign = torch.where(w[expert[bad], :, 20] & 8 > 0, -1.0, 1.0)
        assert torch.equal(out[bad].float(), sign * math.inf)


# -- the least values of each type -----------------------------------------------------------------

LEAST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "e4m3": 2.0 ** -9, "e5m2": 2.0 ** -16}


@pytest.mark.parametrize("want", PATHS)
@pytest.mark.parametrize("kind", [k for k in TYPES if k != "int8"] + ["int4", "e2m1", "int4_f16"])
def test_subnormal_codes(kind, want):
    """Rows of one to three times the type's least value, weights or scales that bring the sums
    back into range: nothing is taken for 0, neither codes nor sums below binary32's normal range."""
    E, BS, N = PATHS[want]
    I, counts = 256, [20, 70, 0, 193] + [0] * (E - 4)
    g = _gen(1)
    w4 = {"int4": "int4", "e2m1": "e2m1", "int4_f16": "int4"}.get(kind)
    rows_kind = kind if not w4 else "f16" if kind == "int4_f16" else "bf16"
    elem = rows_kind.split("_")[-1]
    cfg = cq.make_config(2, E, BS, 1024, 4, token_dtype=int(elem == "f16"))
    assert path(rows_kind, cfg, N, False, w4) == want
    erc, off, ranges = ref.pack_counts(counts, 2)
    cap = cfg.expand_rows_capacity
    x = (_whole((cap, I), -3, 3, g).double() * LEAST[elem]).to(CODES[elem])
    xs, vx = None, x.double()
    if w4:
        w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
        ws = (torch.full((E, N, I // 32), 247, dtype=torch.uint8, device=DEV) if w4 == "e2m1" else
              torch.full((E, N, I // 32), 2.0 ** (120 if elem == "bf16" else 14), device=DEV).to(x.dtype))
        vw = ref.w4_to_f64(w, ws, w4, 32)
        out = cq.grouped_matmul_w4(cfg, cq.make_matmul(I, N, weight_dtype=W4_DTYPE[w4], group_size=32), x, w, ws,
                                   erc.to(DEV), off.to(DEV))
    else:
        wtype = "e4m3" if elem == "e5m2" else elem
        least = {"bf16": 2.0 ** 120, "f16": 2.0 ** 10, "e4m3": 2.0 ** -9}[wtype]
        w = (_whole((E, N, I), -3, 3, g).double() * least).to(CODES[wtype])
        ws = None
        if kind.startswith("mx"):
            xs = torch.full((cap, I // 32), 137, dtype=torch.uint8, device=DEV)
            ws = torch.full((E, N, I // 32), 137, dtype=torch.uint8, device=DEV)
        elif elem in ("e4m3", "e5m2"):
            xs, ws = torch.full((cap,), 1024.0, device=DEV), torch.full((E, N), 1024.0, device=DEV)
        vx, vw = ref.codes_to_f64(x, xs), ref.codes_to_f64(w, ws)
        out = cq.grouped_matmul(cfg, _desc(kind, I, N, False), x, w, erc.to(DEV), off.to(DEV), x_scales=xs,
                                weight_scales=ws)
    for e, (lo, hi) in enumerate(ranges):
        assert torch.equal(out[lo:hi], (vx[lo:hi] @ vw[e].t()).float().to(out.dtype)), e
