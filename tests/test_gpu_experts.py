"""The router and the experts' products on the GPU against plain 64-bit forms (experts_ref)."""
import math

import pytest
import torch

import combine_quant_amd as cq
import experts_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = ("bf16", "f16", "int8", "e4m3", "e5m2", "mx_e4m3", "mx_e5m2")
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(shape, kind, g, x):
    """Random codes of a type (with their natural spread) and their scales, or None."""
    v = torch.randn(shape, generator=g, device=DEV)
    if kind in ("bf16", "f16"):
        return v.to(torch.bfloat16 if kind == "bf16" else torch.float16), None
    if kind == "int8":
        return ((v * 40).round().clamp(-127, 127).to(torch.int8),
                0.01 + torch.rand(shape[:-1], generator=g, device=DEV) * 0.05)
    f8 = F8[kind.split("_")[-1]] if x else torch.float8_e4m3fn
    q = (v * (60 if f8 == torch.float8_e4m3fn else 2000)).to(f8)
    if kind.startswith("mx"):
        s = torch.randint(114, 122, shape[:-1] + (shape[-1] // 32,), generator=g, device=DEV)
        return q, s.to(torch.uint8)
    return q, 0.01 + torch.rand(shape[:-1], generator=g, device=DEV) * 0.05


def _desc(kind, I, N, swiglu):
    x_dtype = {"int8": cq.MOE_DTYPE_INT8, "e4m3": cq.MOE_DTYPE_E4M3, "e5m2": cq.MOE_DTYPE_E5M2,
               "mx_e4m3": cq.MOE_DTYPE_E4M3, "mx_e5m2": cq.MOE_DTYPE_E5M2}.get(kind, 0)
    scaling = (cq.MOE_MM_SCALE_MX if kind.startswith("mx") else
               cq.MOE_MM_SCALE_ROW if x_dtype else cq.MOE_MM_SCALE_NONE)
    return cq.make_matmul(I, N, x_dtype=x_dtype, scaling=scaling,
                          activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)


def _config(W, counts, H=1024, f16=False, extra=5):
    """A config with room for the rows (and `extra` more) of these per-expert counts."""
    total = sum(counts)
    K = min(16, len(counts))
    bs = max(1, -(-total // (W * K)))
    assert bs <= 512
    return cq.make_config(W, len(counts), bs, H, K, cap=W * bs * K + extra,
                          token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)


def _run_product(kind, W, counts, I, N, swiglu, seed=0):
    g = _gen(seed)
    cfg = _config(W, counts, f16=kind == "f16")
    cap, rows = cfg.expand_rows_capacity, sum(counts)
    erc, off, ranges = ref.pack_counts(counts, W)
    x, xs = _codes((cap, I), kind, g, True)
    w, ws = _codes((len(counts), N, I), kind, g, False)
    if kind in ("bf16", "f16"):
        w = (w.float() / math.sqrt(I)).to(w.dtype)
    elif xs.dtype == torch.float32:
        # outputs near 1: scales that undo the codes' own magnitude
        ws *= 2.0 ** -round(math.log2(x[:, :32].float().abs().mean() * w.float().abs().mean()
                                      * math.sqrt(I) * 0.0016))
    else:
        drop = round(math.log2(x[:, :32].float().abs().mean() * w.float().abs().mean()
                               * math.sqrt(I))) - 18
        ws = (ws.int() - drop).clamp(1, 254).to(torch.uint8)
    if rows < cap:                     # what lies behind the last row must not matter
        bits = x.view(torch.uint8) if x.element_size() == 1 else x.view(torch.int16)
        bits[rows:] = 0x7F if x.element_size() == 1 else 0x7FFF       # NaN in the float types
    out = torch.full((cap, N // 2 if swiglu else N), 7.25, device=DEV,
                     dtype=torch.float16 if kind == "f16" else torch.bfloat16)
    cq.grouped_matmul(cfg, _desc(kind, I, N, swiglu), x, w, erc.to(DEV), off.to(DEV),
                      x_scales=xs, weight_scales=ws, out=out)
    torch.cuda.synchronize()
    y, err = ref.product(ref.codes_to_f64(x[:rows], None if xs is None else xs[:rows]),
                         ref.codes_to_f64(w, ws), ranges, swiglu, cut="e4m3" in kind or "e5m2" in kind)
    ref.check(out, y, err, rows)
    assert (out[rows:] == 7.25).all()


COUNTS = [
    (2, [0, 0, 1, 0]),                                  # a single row
    (2, [0, 0, 0, 0]),                                  # none at all
    (3, [1, 2, 15, 16, 17, 0]),
    (2, [31, 33, 64, 65, 0, 7, 100, 129]),
    (2, [0, 260, 0, 127]),
    (5, [300, 3, 0, 0, 513]),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("W,counts", COUNTS)
def test_product_row_counts(kind, W, counts, swiglu):
    _run_product(kind, W, counts, 256, 160, swiglu, seed=len(counts))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("I,N,swiglu", [
    (0, 2, True), (0, 1, False), (1, 33, False), (2, 777, False), (3, 258, True), (9, 130, True),
    (17, 514, True), (33, 1000, False),
])
def test_product_odd_sizes(kind, I, N, swiglu):
    """Inner sizes of I + 1 steps of the type's granularity (chunks that end inside a tile)."""
    step = 128 if kind.startswith("mx") else 8 if kind in ("bf16", "f16") else 16
    _run_product(kind, 2, [5, 0, 90, 21], step * (I + 1), N, swiglu, seed=I)


@pytest.mark.parametrize("kind", TYPES)
def test_product_many_rows(kind):
    """Enough rows per expert for the large tiles, ragged ends included."""
    _run_product(kind, 2, [700, 0, 257, 512, 1, 1025, 385, 255], 896, 520, True, seed=5)
    _run_product(kind, 2, [513, 1281, 0, 2], 640, 1029, False, seed=6)


# Rows per expert that give every tile height, several tiles per expert and empty experts; with 32
# experts and more than 1536 weight rows there are tiles enough for the tile kernels.
RAGGED = [0, 1, 33, 64, 65, 97, 130, 161, 193, 225, 256, 257, 300, 511, 513, 769,
          31, 32, 0, 0, 16, 15, 2, 90, 224, 128, 129, 5, 48, 70, 0, 449]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("steps,N,swiglu", [
    (0, 1600, False), (1, 1666, True), (2, 1541, False), (8, 1602, True), (25, 1537, False),
    (40, 2054, True),
])
def test_product_tiles(kind, steps, N, swiglu):
    """Inner sizes of steps + 1 pieces of the type's granularity through the tile kernels."""
    step = 128 if kind.startswith("mx") else 24 if kind in ("bf16", "f16") else 48
    _run_product(kind, 4, RAGGED, step * (steps + 1), N, swiglu, seed=steps)


@pytest.mark.parametrize("kind", ["int8", "e4m3", "e5m2"])
def test_product_without_row_scales(kind):
    """x_scales may be absent (static quantization): every row scale is 1."""
    counts, W, I, N = [3, 40, 0, 9], 2, 128, 48
    cfg = _config(W, counts, extra=0)
    g = _gen(1)
    erc, off, ranges = ref.pack_counts(counts, W)
    x, _ = _codes((cfg.expand_rows_capacity, I), kind, g, True)
    w, ws = _codes((4, N, I), kind, g, False)
    out = cq.grouped_matmul(cfg, _desc(kind, I, N, False), x, w, erc.to(DEV), off.to(DEV),
                            weight_scales=ws)
    y, err = ref.product(x[:52].double(), ref.codes_to_f64(w, ws), ranges, False,
                         cut=kind != "int8")
    ref.check(out, y, err, 52)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "mx_e4m3"])
def test_nan_and_infinity_stay_in_their_row(kind):
    counts, W, I, N = [20, 70, 0, 300], 2, 256, 64
    cfg = _config(W, counts, extra=0)
    g = _gen(2)
    erc, off, ranges = ref.pack_counts(counts, W)
    rows = sum(counts)
    x, xs = _codes((cfg.expand_rows_capacity, I), kind, g, True)
    w, ws = _codes((4, N, I), kind, g, False)
    mm = _desc(kind, I, N, False)
    args = (mm, x, w, erc.to(DEV), off.to(DEV))
    clean = cq.grouped_matmul(cfg, *args, x_scales=xs, weight_scales=ws).clone()
    bad = [0, 19, 25, 90, 389]
    x.view(torch.uint8 if kind != "bf16" else torch.int16)[bad, 13] = 0x7F if kind != "bf16" else 0x7FC0
    dirty = cq.grouped_matmul(cfg, *args, x_scales=xs, weight_scales=ws)
    hit = torch.zeros(cfg.expand_rows_capacity, dtype=torch.bool, device=DEV)
    hit[bad] = True
    assert torch.isnan(dirty[:rows][hit[:rows]].float()).all()
    assert torch.equal(dirty[:rows][~hit[:rows]], clean[:rows][~hit[:rows]])


@pytest.mark.parametrize("kind,rows", [("e4m3", 3), ("e4m3", 300), ("bf16", 3)])
def test_weights_past_32_bits(kind, rows):
    """Weights of more than 2^32 bytes: the last expert's products are right."""
    W, E, I, N = 2, 70, 8192, 8192 if kind == "e4m3" else 4096
    counts = [0] * (E - 1) + [rows]
    cfg = _config(W, counts, extra=0)
    g = _gen(3)
    erc, off, ranges = ref.pack_counts(counts, W)
    x, xs = _codes((cfg.expand_rows_capacity, I), kind, g, True)
    w1, ws1 = _codes((N, I), kind, g, False)
    w = torch.empty((E, N, I), dtype=w1.dtype, device=DEV)
    w[E - 1] = w1
    assert w.numel() * w.element_size() > 2 ** 32
    ws = None
    if ws1 is not None:
        ws = torch.zeros((E, N), device=DEV)
        ws[E - 1] = ws1 * 1e-4
        ws1 = ws[E - 1]
    out = cq.grouped_matmul(cfg, _desc(kind, I, N, False), x, w, erc.to(DEV), off.to(DEV),
                            x_scales=xs, weight_scales=ws)
    y, err = ref.product(ref.codes_to_f64(x[:rows], None if xs is None else xs[:rows]),
                         ref.codes_to_f64(w1, ws1)[None], [(0, rows)], False, cut=kind == "e4m3")
    ref.check(out, y, err, rows)


# -- 4-bit weights ------------------------------------------------------------------------------

def _run_w4(token, weight, group, W, counts, I, N, swiglu, seed=0):
    g = _gen(seed)
    f16 = token == "f16"
    dt = torch.float16 if f16 else torch.bfloat16
    cfg = _config(W, counts, f16=f16)
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    erc, off, ranges = ref.pack_counts(counts, W)
    x = torch.randn((cap, I), generator=g, device=DEV).to(dt)
    x[rows:] = float("nan")
    w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    if weight == "int4":
        ws = ((0.5 + torch.rand((E, N, I // group), generator=g, device=DEV)) / (4.6 * math.sqrt(I))).to(dt)
        surplus = 288.0 * ws.double().repeat_interleave(group, 2)     # |136 x| twice, + |code x|
    else:
        ws = torch.randint(119, 124, (E, N, I // group), generator=g, device=DEV).to(torch.uint8)
        surplus = None
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_INT4 if weight == "int4" else cq.MOE_W4_E2M1,
                        group_size=group,
                        activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)
    out = torch.full((cap, N // 2 if swiglu else N), 7.25, device=DEV, dtype=dt)
    cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV), out=out)
    torch.cuda.synchronize()
    values = ref.w4_to_f64(w, ws, weight, group)
    if f16 or weight == "e2m1":
        surplus = None                                                # codes enter as they are
    if surplus is not None:
        # Only the sum inside one group meets the surplus: its (group + 16) roundings, seen
        # over the whole row's bound of (I + 16), plus the ordinary terms.
        surplus = surplus * (group + 16) / (I + 16) + values.abs()
    y, err = ref.product(x[:rows].double(), values, ranges, swiglu, surplus)
    ref.check(out, y, err, rows)
    assert (out[rows:] == 7.25).all()


W4 = [("int4", 32), ("int4", 64), ("int4", 128), ("e2m1", 32)]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("W,counts", COUNTS)
def test_4bit_row_counts(token, weight, group, W, counts, swiglu):
    _run_w4(token, weight, group, W, counts, 256, 160, swiglu, seed=len(counts))


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("I,N,swiglu", [
    (0, 2, True), (0, 1, False), (1, 33, False), (2, 777, False), (4, 258, True), (20, 514, True),
])
def test_4bit_odd_sizes(token, weight, group, I, N, swiglu):
    _run_w4(token, weight, group, 2, [5, 0, 90, 21], group * (I + 1), N, swiglu, seed=I)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
def test_4bit_many_rows(token, weight, group):
    _run_w4(token, weight, group, 2, [700, 0, 257, 512, 1, 1025, 385, 255], 896, 520, True, seed=5)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("groups,N,swiglu", [
    (1, 1600, False), (2, 1666, True), (3, 1541, False), (7, 1602, True), (13, 1537, False),
    (20, 2054, True),
])
def test_4bit_tiles(token, weight, group, groups, N, swiglu):
    _run_w4(token, weight, group, 4, RAGGED, group * groups, N, swiglu, seed=groups)


# A few rows per expert on many experts: the tiles of one decode step (one expert has a prompt's).
FEW = [1, 0, 2, 33, 16, 17, 0, 5, 1, 1, 31, 32, 3, 70, 0, 8, 4, 12, 15, 64, 2, 2, 0, 9, 24, 25, 6, 7, 1, 0, 11, 130]


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("weight,group", W4)
@pytest.mark.parametrize("groups,N,swiglu", [
    (1, 1600, False), (2, 1666, True), (5, 1541, False), (9, 1602, True), (24, 1537, False),
])
def test_4bit_few_rows(token, weight, group, groups, N, swiglu):
    _run_w4(token, weight, group, 4, FEW, group * groups, N, swiglu, seed=groups)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("steps,N,swiglu", [(0, 1600, False), (3, 1666, True), (30, 1541, False)])
def test_product_few_rows(kind, steps, N, swiglu):
    step = 128 if kind.startswith("mx") else 24 if kind in ("bf16", "f16") else 48
    _run_product(kind, 4, FEW, step * (steps + 1), N, swiglu, seed=steps)


def test_4bit_every_code():
    """Each code alone against a one-hot row gives code * scale exactly."""
    for token, weight, group in (("bf16", "int4", 32), ("f16", "int4", 32), ("bf16", "e2m1", 32),
                                 ("f16", "e2m1", 32)):
        dt = torch.float16 if token == "f16" else torch.bfloat16
        I, N, W, counts = 128, 16, 2, [128, 0]
        cfg = _config(W, counts, f16=token == "f16", extra=0)
        erc, off, _ = ref.pack_counts(counts, W)
        x = torch.zeros((cfg.expand_rows_capacity, I), dtype=dt, device=DEV)
        x[torch.arange(128), torch.arange(128)] = 1.0
        g = _gen(4)
        w = torch.randint(0, 256, (2, N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
        w[0, :, 0] = torch.arange(16, device=DEV) * 17
        if weight == "int4":
            ws = torch.full((2, N, I // group), 0.5, dtype=dt, device=DEV)
        else:
            ws = torch.full((2, N, I // group), 126, dtype=torch.uint8, device=DEV)
        mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_INT4 if weight == "int4" else
                            cq.MOE_W4_E2M1, group_size=group)
        out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))
        assert torch.equal(out[:128].double(), ref.w4_to_f64(w, ws, weight, group)[0].t())


def _check_extremes(out, x, w, ranges, rows):
    """x and w are not negative, so no partial sum exceeds the result: above fp32's range it is
    infinite, and below it the usual bound holds, with 2^-125 more where the result or its last
    sum may be subnormal (2^-126 in the sum, and as much in the rounding)."""
    y, err = ref.product(x, w, ranges, False, cut=True)
    got = out[:rows].double()
    nan = torch.isnan(y)
    assert nan.any() and torch.equal(torch.isnan(got), nan)
    big = y >= 2.0 ** 128
    assert big.any() and torch.isinf(got[big]).all()
    rest = y < 2.0 ** 127
    tol = err + 2.0 ** -8 * (y + err) + 2.0 ** -125
    assert (y[rest] < 2.0 ** -100).any() and ((got - y).abs()[rest] <= tol[rest]).all()


@pytest.mark.parametrize("counts,N", [([60, 0, 29, 5], 70), ([70, 0, 129, 5] * 8, 1600)])
def test_mx_scales_to_the_ends_of_their_range(counts, N):
    W, I = 2, 256
    cfg = _config(W, counts, extra=0)
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    g = _gen(11)
    erc, off, ranges = ref.pack_counts(counts, W)
    x = torch.rand((cap, I), generator=g, device=DEV).add(0.1).to(torch.float8_e4m3fn)
    w = torch.rand((E, N, I), generator=g, device=DEV).add(0.1).to(torch.float8_e4m3fn)
    ends = torch.tensor([0, 1, 2, 40, 64, 100, 127, 150, 190, 220, 253, 254, 255], device=DEV, dtype=torch.uint8)
    xs = ends[torch.arange(cap, device=DEV) % 13][:, None].expand(cap, I // 32).contiguous()
    ws = ends[torch.arange(E * N, device=DEV) % 13].view(E, N, 1).expand(E, N, I // 32).contiguous()
    out = cq.grouped_matmul(cfg, _desc("mx_e4m3", I, N, False), x, w, erc.to(DEV), off.to(DEV),
                            x_scales=xs, weight_scales=ws)
    nan = float("nan")
    vx = ref.codes_to_f64(x, xs).masked_fill((xs == 255)[:, :1], nan)[:rows]
    vw = ref.codes_to_f64(w, ws).masked_fill((ws == 255)[:, :, :1], nan)
    _check_extremes(out, vx, vw, ranges, rows)


@pytest.mark.parametrize("counts,N", [([60, 0, 29, 5], 70), ([70, 0, 129, 5] * 8, 1600),
                                      ([16, 0, 9, 5] * 8, 1600)])
def test_e2m1_scales_to_the_ends_of_their_range(counts, N):
    W, I = 2, 256
    cfg = _config(W, counts, extra=0)
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    g = _gen(12)
    erc, off, ranges = ref.pack_counts(counts, W)
    ends = torch.tensor([0, 1, 2, 3, 40, 64, 100, 127, 150, 190, 220, 252, 255], device=DEV, dtype=torch.uint8)
    powers = torch.tensor([-100, -60, 0, 3, 60, 110], device=DEV)[torch.arange(cap, device=DEV) % 6]
    x = torch.rand((cap, I), generator=g, device=DEV).add(0.1).mul(2.0 ** powers[:, None]).bfloat16()
    w = torch.randint(0, 256, (E, N, I // 2), generator=g, device=DEV, dtype=torch.uint8) & 0x77
    ws = ends[torch.arange(E * N, device=DEV) % 13].view(E, N, 1).expand(E, N, I // 32).contiguous()
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_E2M1, group_size=32)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))
    vw = ref.w4_to_f64(w, ws, "e2m1", 32).masked_fill((ws == 255)[:, :, :1], float("nan"))
    _check_extremes(out, x[:rows].double(), vw, ranges, rows)


@pytest.mark.parametrize("token", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64])
def test_4bit_infinite_last_scale(token, group):
    """The last group of a row that ends inside a chunk of 128 has an infinite scale."""
    dt = torch.float16 if token == "f16" else torch.bfloat16
    W, counts, N, I = 2, [5, 0, 18, 2], 33, 128 + group
    cfg = _config(W, counts, f16=token == "f16", extra=0)
    erc, off, _ = ref.pack_counts(counts, W)
    x = torch.ones((cfg.expand_rows_capacity, I), dtype=dt, device=DEV)
    w = torch.full((4, N, I // 2), 0x11, dtype=torch.uint8, device=DEV)
    w[:, 1::2] = 0xFF                                                # -1
    ws = torch.ones((4, N, I // group), dtype=dt, device=DEV)
    ws[..., -1] = float("inf")
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_INT4, group_size=group)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))[:25].float()
    assert (out[:, ::2] == float("inf")).all() and (out[:, 1::2] == -float("inf")).all()


def test_4bit_weights_past_32_bits():
    W, E, I, N = 2, 140, 8192, 8192
    counts = [0] * (E - 1) + [2]
    cfg = _config(W, counts, extra=0)
    g = _gen(3)
    erc, off, _ = ref.pack_counts(counts, W)
    x = torch.randn((cfg.expand_rows_capacity, I), generator=g, device=DEV).bfloat16()
    w = torch.empty((E, N, I // 2), dtype=torch.uint8, device=DEV)
    w[-1] = torch.randint(0, 256, (N, I // 2), generator=g, device=DEV, dtype=torch.uint8)
    ws = torch.full((E, N, I // 32), 120, dtype=torch.uint8, device=DEV)
    assert w.numel() > 2 ** 32
    mm = cq.make_matmul(I, N, weight_dtype=cq.MOE_W4_E2M1, group_size=32)
    out = cq.grouped_matmul_w4(cfg, mm, x, w, ws, erc.to(DEV), off.to(DEV))
    y, err = ref.product(x[:2].double(), ref.w4_to_f64(w[-1:], ws[-1:], "e2m1", 32), [(0, 2)], False)
    ref.check(out, y, err, 2)


# -- the router ---------------------------------------------------------------------------------

def _run_gate(W, BS, E, Z, K, logits, bias, sigmoid=False, groups=1, keep=1, top=1, renorm=False,
              factor=1.0):
    cfg = cq.make_config(W, E, BS, 1024, K, zero_expert_num=Z)
    gate = cq.make_gate(cq.MOE_SCORE_SIGMOID if sigmoid else cq.MOE_SCORE_SOFTMAX, groups, keep,
                        top, renorm, factor)
    n = E + Z
    ids, w = cq.gate_topk(cfg, gate, logits.view(W, BS, n).to(DEV),
                          None if bias is None else bias.to(DEV))
    rid, rw = ref.gate(logits.view(-1, n), bias, K, sigmoid, groups, keep, top, renorm, factor)
    assert torch.equal(ids.view(-1, K).cpu(), rid)
    # formed in binary64, rounded once to fp32
    diff = (w.view(-1, K).cpu().double() - rw).abs()
    assert (diff <= 2.0 ** -23 * rw.abs() + 2.0 ** -149).all(), float(diff.max())


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("W,BS,E,Z,K,groups,keep,top", [
    (2, 1, 8, 0, 2, 1, 1, 1), (2, 3, 256, 0, 8, 8, 4, 2), (2, 5, 256, 0, 8, 8, 3, 1),
    (3, 7, 15, 2, 4, 1, 1, 1), (4, 2, 64, 1, 16, 5, 2, 2), (2, 9, 512, 4, 16, 1, 1, 1),
    (2, 2, 1024, 1024, 16, 64, 1, 2), (5, 33, 60, 0, 1, 60, 1, 1), (2, 4, 640, 1, 7, 1, 1, 1),
])
def test_router(W, BS, E, Z, K, groups, keep, top, with_bias, sigmoid):
    g = torch.Generator().manual_seed(W * 100 + K)
    n = E + Z
    logits = torch.randn((W * BS, n), generator=g) * 2
    bias = torch.randn((n,), generator=g) * 0.1 if with_bias else None
    _run_gate(W, BS, E, Z, K, logits, bias, sigmoid, groups, keep, top, True, 2.5)
    _run_gate(W, BS, E, Z, K, logits, bias, sigmoid, groups, keep, top, False, 1.0)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("W,BS,E,Z,K,groups,keep,top", [
    (4, 512, 256, 0, 8, 8, 4, 2), (16, 131, 16, 0, 3, 1, 1, 1), (8, 300, 512, 4, 16, 1, 1, 1),
    (5, 411, 180, 1, 16, 1, 1, 1), (4, 512, 252, 4, 12, 64, 20, 1), (8, 257, 576, 0, 9, 18, 5, 2),
])
def test_router_many_tokens(W, BS, E, Z, K, groups, keep, top, with_bias, sigmoid):
    """Tokens enough for four to share a wave, the last wave partly empty."""
    g = torch.Generator().manual_seed(W + K)
    n = E + Z
    logits = torch.randn((W * BS, n), generator=g) * 2
    logits[::7] = (logits[::7] * 4).round() / 4                 # many equal logits in some rows
    bias = torch.randn((n,), generator=g) * 0.1 if with_bias else None
    _run_gate(W, BS, E, Z, K, logits, bias, sigmoid, groups, keep, top, True, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (8, 3, 2), (4, 2, 1)])
def test_router_ties_go_to_the_lower_id(sigmoid, groups, keep, top):
    g = torch.Generator().manual_seed(9)
    logits = torch.randint(-2, 3, (64, 128), generator=g).float()
    bias = torch.randint(0, 2, (128,), generator=g).float() * 0.25
    for b in (None, bias):
        _run_gate(2, 32, 128, 0, 8, logits, b, sigmoid, groups, keep, top, True, 1.0)
    _run_gate(2, 32, 128, 0, 8, torch.zeros((64, 128)), None, sigmoid, groups, keep, top, True, 1.0)


def test_router_orders_choices_that_agree_in_32_bits():
    """Sigmoid scores far closer together than a step of binary32 keep their order."""
    n = 256
    z = torch.full((8, n), 14.0)
    z += torch.arange(n).flip(0).float()[None, :] * 2.0 ** -20 * torch.arange(1, 9)[:, None]
    bias = torch.zeros(n)
    _run_gate(2, 4, n, 0, 8, z, bias, True, 1, 1, 1, True, 1.0)
    _run_gate(2, 4, n, 0, 8, z.flip(1).contiguous(), bias, True, 8, 4, 2, True, 1.0)


def test_router_masked_rows():
    """Rows of -infinity, of the lowest finite value, and with NaN keep ids distinct."""
    low = torch.finfo(torch.float32).min
    z = torch.zeros((6, 64))
    z[0] = -math.inf
    z[1] = low
    z[2] = -math.inf
    z[2, 40] = 1.0
    z[3, ::2] = -math.inf
    z[4, 3:7] = math.nan
    z[5] = math.nan
    cfg = cq.make_config(2, 64, 3, 1024, 4)
    for score in (cq.MOE_SCORE_SOFTMAX, cq.MOE_SCORE_SIGMOID):
        for bias in (None, torch.zeros(64, device=DEV)):
            for groups in (1, 4):
                gate = cq.make_gate(score, groups, groups, 1, True)
                ids, w = cq.gate_topk(cfg, gate, z.view(2, 3, 64).to(DEV), bias)
                ids, w = ids.view(6, 4).cpu(), w.view(6, 4).cpu()
                assert ((ids >= 0) & (ids < 64)).all()
                assert all(len(set(r)) == 4 for r in ids.tolist())
                assert (w[0] == 0).all()
                assert ids[2, 0] == 40 and w[2, 0] == 1.0 and (w[2, 1:] == 0).all()
                assert ids[3].tolist() == [1, 3, 5, 7]
                if score == cq.MOE_SCORE_SIGMOID:
                    assert ids[4].tolist() == [0, 1, 2, 7]
                else:
                    assert ids[1].tolist() == [0, 1, 2, 3] and (w[1] == 0.25).all()


def test_router_infinite_biases():
    """A group whose two best choices are infinities of both signs has no value: it comes last."""
    z = torch.randn((6, 64), generator=torch.Generator().manual_seed(3))
    bias = torch.full((64,), -math.inf)
    bias[16:32] = 0.0
    bias[3] = math.inf
    cfg = cq.make_config(2, 64, 3, 1024, 4)
    for score in (cq.MOE_SCORE_SOFTMAX, cq.MOE_SCORE_SIGMOID):
        gate = cq.make_gate(score, 4, 1, 2, True)
        ids, w = cq.gate_topk(cfg, gate, z.view(2, 3, 64).to(DEV), bias.to(DEV))
        ids = ids.view(6, 4).cpu()
        assert torch.equal(ids.long(), z[:, 16:32].topk(4, 1).indices + 16)
        assert torch.isfinite(w).all()


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("W,BS", [(2, 1), (8, 275)])
def test_router_scores_over_the_whole_range(W, BS, renorm):
    """Sigmoids from 0 over subnormal binary32 values to 1; the biases alone decide the order."""
    z = torch.tensor([-1e30, -800.0, -745.0, -103.5, -100.0, -90.0, -40.0, -16.0, -1.0, -1e-30, 0.0,
                      1e-6, 1.0, 20.0, 90.0, 1e30])
    g = torch.Generator().manual_seed(5)
    logits = torch.stack([z[torch.randperm(16, generator=g)] for _ in range(W * BS)])
    bias = torch.randperm(16, generator=g).float() * 4
    _run_gate(W, BS, 16, 0, 16, logits, bias, True, 1, 1, 1, renorm, 1.0)
    _run_gate(W, BS, 16, 0, 16, logits / 8, bias, False, 1, 1, 1, renorm, 1.0)
