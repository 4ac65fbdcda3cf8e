"""The products of block-scaled rows on the GPU, with tokens or codes as results, against plain
64-bit forms (block_ref)."""
import math

import pytest
import torch

import block_ref as blk
import combine_quant_amd as cq
import experts_path
import experts_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
KINDS = ("e4m3", "e5m2")
CODE = {"e4m3": cq.MOE_DTYPE_E4M3, "e5m2": cq.MOE_DTYPE_E5M2}
experts_path.TYPES.update(block_e4m3=7, block_e5m2=8)
experts_path.NAMES = experts_path.NAMES[:3] + ("thin",)


def _config(W, counts, f16=False, extra=5):
    total = sum(counts)
    K = min(16, len(counts))
    bs = max(1, -(-total // (W * K)))
    assert bs <= 512
    return cq.make_config(W, len(counts), bs, 1024, K, cap=W * bs * K + extra,
                          token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)


def _desc(kind, I, N, swiglu):
    return cq.make_matmul(I, N, x_dtype=CODE[kind], scaling=cq.MOE_MM_SCALE_BLOCK,
                          activation=cq.MOE_ACT_SWIGLU if swiglu else cq.MOE_ACT_NONE)


def _case(kind, W, counts, I, N, swiglu, seed, f16=False, cut=True):
    """Config, descriptor, tensors and the 64-bit result with its bound.  Results near 1."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cfg = _config(W, counts, f16)
    cap, rows, E = cfg.expand_rows_capacity, sum(counts), len(counts)
    parts = 2 if swiglu else 1
    erc, off, ranges = ref.pack_counts(counts, W)
    x = (torch.randn((cap, I), generator=g, device=DEV) * blk.TOP[kind] / 8).to(blk.F8[kind])
    w = (torch.randn((E, N, I), generator=g, device=DEV) * 60).to(torch.float8_e4m3fn)
    xs = (0.2 + torch.rand((cap, blk.groups(I)), generator=g, device=DEV)) * 8 / blk.TOP[kind]
    ws = (0.2 + torch.rand((E, parts * blk.groups(N // parts), blk.groups(I)), generator=g, device=DEV)) / (
        60 * math.sqrt(I))
    x.view(torch.uint8)[rows:] = 0x7F                      # NaN behind the last row
    xs[rows:] = math.nan
    y, err = blk.product(x[:rows], xs[:rows], w, ws, ranges, swiglu, cut)
    return cfg, _desc(kind, I, N, swiglu), x, xs, w, ws, erc.to(DEV), off.to(DEV), y, err


def _run(kind, W, counts, I, N, swiglu, seed=0, f16=False):
    cfg, mm, x, xs, w, ws, erc, off, y, err = _case(kind, W, counts, I, N, swiglu, seed, f16)
    rows = sum(counts)
    out = torch.full((cfg.expand_rows_capacity, y.shape[1]), 7.25, device=DEV,
                     dtype=torch.float16 if f16 else torch.bfloat16)
    cq.grouped_matmul(cfg, mm, x, w, erc, off, x_scales=xs, weight_scales=ws, out=out)
    torch.cuda.synchronize()
    ref.check(out, y, err, rows)
    assert (out[rows:] == 7.25).all()


def _run_codes(kind, to, W, counts, I, N, swiglu, seed=0):
    # up to 64 rows a tile the products are whole
    cfg, mm, x, xs, w, ws, erc, off, y, err = _case(kind, W, counts, I, N, swiglu, seed, cut=max(counts) > 64)
    rows, M = sum(counts), y.shape[1]
    codes = torch.full((cfg.expand_rows_capacity, M), 0x55, device=DEV, dtype=torch.uint8)
    scales = torch.full((cfg.expand_rows_capacity, blk.groups(M)), 7.25, device=DEV)
    cq.grouped_matmul_quantize(cfg, mm, CODE[to], x, xs, w, ws, erc, off, out=(codes, scales))
    torch.cuda.synchronize()
    blk.check_codes(codes.view(blk.F8[to]), scales, y, err, to, rows)
    assert (codes[rows:] == 0x55).all() and (scales[rows:] == 7.25).all()


COUNTS = [
    (2, [0, 0, 1, 0]),
    (2, [0, 0, 0, 0]),
    (3, [1, 2, 15, 16, 17, 0]),
    (2, [31, 33, 64, 65, 0, 7, 100, 129]),
    (5, [300, 3, 0, 0, 513]),
]
FEW = (2, [0, 3, 17, 50])                               # 18 rows an expert: streamed
SOME = (2, [0, 3, 17, 65, 200, 0])                      # 48: thin tiles
MANY = (2, [(7 * e) % 5 for e in range(254)] + [193, 400])       # 256 experts: large tiles


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("W,counts", COUNTS)
def test_row_counts(kind, W, counts, swiglu):
    _run(kind, W, counts, 272, 320, swiglu, seed=len(counts))


SIZES = [(16, 1, False), (16, 2, True), (112, 33, False), (128, 256, True), (144, 129, False),
         (368, 258, True), (384, 127, False), (496, 62, True), (512, 385, False), (528, 514, True),
         (640, 512, False), (1136, 777, False), (1280, 1000, True)]


ROUTES = [(*FEW, "stream"), (*SOME, "thin"), (*MANY, "tiles")]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("I,N,swiglu", SIZES)
@pytest.mark.parametrize("W,counts,path", ROUTES)
def test_sizes(W, counts, path, I, N, swiglu, kind):
    assert experts_path.path("block_" + kind, _config(W, counts), N, swiglu) == path
    _run(kind, W, counts, I, N, swiglu, seed=I + N, f16=N % 2 == 0)


@pytest.mark.parametrize("kind,to", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("I,N,swiglu", SIZES)
def test_codes_sizes(kind, to, I, N, swiglu):
    _run_codes(kind, to, 2, [0, 3, 17, 50], I, N, swiglu, seed=I + N)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("W,counts", COUNTS + [SOME, MANY])
def test_codes_row_counts(W, counts, swiglu):
    _run_codes("e4m3", "e4m3", W, counts, 272, 320, swiglu, seed=len(counts))


@pytest.mark.parametrize("coded", [False, True])
def test_every_tile_height(coded):
    """Large tiles of 1 to 14 times 16 rows."""
    counts = [16 * h - h % 3 for h in range(1, 15)] + [1] * 242
    assert experts_path.path("block_e4m3", _config(2, counts), 256, True) == "tiles"
    if coded:
        _run_codes("e4m3", "e4m3", 2, counts, 400, 256, True, seed=1)
    else:
        _run("e4m3", 2, counts, 400, 256, True, seed=1)


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("E", [130, 512, 1024])
def test_thin_tiles_of_many_experts(E, coded):
    counts = [0] * E
    for e in range(0, E, E // 36):
        counts[e] = 1 + e % 3
    counts[E - 1] = 70
    cfg = _config(2, counts)
    N = 128
    assert experts_path.path("block_e4m3", cfg, N, False) == "thin"
    if coded:
        _run_codes("e4m3", "e5m2", 2, counts, 272, N, False, seed=E)
    else:
        _run("e4m3", 2, counts, 272, N, False, seed=E)


@pytest.mark.parametrize("I,N,swiglu,counts", [
    (65536, 40, False, [3, 0, 1, 2]), (65536, 300, True, [0, 40, 200, 70]), (16, 65536, False, [1, 0, 2, 0]),
    (48, 65536, True, [30, 0, 0, 65]), (32768, 1024, False, [9, 8, 7, 0])])
def test_largest_sizes(I, N, swiglu, counts):
    _run("e4m3", 2, counts, I, N, swiglu, seed=3)
    _run_codes("e4m3", "e4m3", 2, counts, I, N, swiglu, seed=3)


def _exact_case(counts, I, N, seed):
    """Small whole codes and scales that are powers of two: every sum is exact in fp32."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    cfg = _config(2, counts, extra=0)
    cap, E = cfg.expand_rows_capacity, len(counts)
    whole = lambda *n: torch.randint(-3, 4, n, generator=g, device=DEV).float()  # noqa: E731
    x, w = whole(cap, I).to(torch.float8_e4m3fn), whole(E, N, I).to(torch.float8_e4m3fn)
    power = lambda *n: 2.0 ** torch.randint(-1, 2, n, generator=g, device=DEV).float()  # noqa: E731
    return cfg, x, power(cap, blk.groups(I)), w, power(E, blk.groups(N), blk.groups(I))


@pytest.mark.parametrize("counts,path", [([5, 0, 33, 64], "stream"), (SOME[1], "thin"), (MANY[1], "tiles")])
@pytest.mark.parametrize("I,N", [(48, 200), (640, 150), (1040, 256)])
def test_every_scale_meets_its_block(counts, path, I, N):
    cfg, x, xs, w, ws = _exact_case(counts, I, N, I + N)
    assert experts_path.path("block_e4m3", cfg, N, False) == path
    erc, off, ranges = ref.pack_counts(counts, 2)
    out = cq.grouped_matmul(cfg, _desc("e4m3", I, N, False), x, w, erc.to(DEV), off.to(DEV),
                            x_scales=xs, weight_scales=ws)
    torch.cuda.synchronize()
    rows = sum(counts)
    y, _ = blk.product(x[:rows], xs[:rows], w, ws, ranges, False)
    assert (out[:rows] == y.to(torch.float32).to(torch.bfloat16)).all()


@pytest.mark.parametrize("counts", [[5, 0, 33, 64], SOME[1], MANY[1]])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_bad_scales_stay_in_their_row_and_block(counts, bad):
    I, N = 400, 300
    cfg, x, xs, w, ws = _exact_case(counts, I, N, 5)
    erc, off, ranges = ref.pack_counts(counts, 2)
    call = lambda: cq.grouped_matmul(cfg, _desc("e4m3", I, N, False), x, w, erc.to(DEV),  # noqa: E731
                                     off.to(DEV), x_scales=xs, weight_scales=ws)
    rows = sum(counts)
    good = call()[:rows].clone()
    xs[2, 3] = bad                                         # row 2, its last and short group
    e = max(i for i, r in enumerate(ranges) if r[1] > r[0])
    ws[e, 1, 0] = bad                                      # columns 128..255 of the last expert
    out = call()[:rows]
    lo, hi = ranges[e]
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[2] = True
    hit[lo:hi, 128:256] = True
    assert (out[~hit] == good[~hit]).all()
    assert not torch.isfinite(out[2]).any() and not torch.isfinite(out[lo:hi, 128:256]).any()


def test_codes_of_groups_that_are_zero_or_not_finite():
    I, N, counts = 256, 320, [5, 0, 33, 64]
    cfg, x, xs, w, ws = _exact_case(counts, I, N, 6)
    erc, off, _ = ref.pack_counts(counts, 2)
    call = lambda: cq.grouped_matmul_quantize(cfg, _desc("e4m3", I, N, False), CODE["e4m3"], x, xs,  # noqa: E731
                                              w, ws, erc.to(DEV), off.to(DEV))
    good, gs = (t.clone() for t in call())
    xs[1] = 0.0
    xs[7, 1] = math.inf
    ws[3, 2] = math.nan                                    # columns 256..319 of the last expert
    codes, s = call()
    rows = sum(counts)
    assert (codes[1] & 0x7F == 0).all() and (s[1] == 0).all()
    assert (codes[7] == 0).all() and s[7].isnan().all()
    assert (codes[38:rows, 256:] == 0).all() and s[38:rows, 2].isnan().all()
    keep = [0] + list(range(2, 7)) + list(range(8, 38))
    assert (codes[keep] == good[keep]).all() and (s[keep] == gs[keep]).all()
    assert (codes[38:rows, :256] == good[38:rows, :256]).all() and (s[38:rows, :2] == gs[38:rows, :2]).all()


@pytest.mark.parametrize("counts", [[5, 0, 33, 64], SOME[1], MANY[1]])
def test_same_bytes_every_time(counts):
    cfg, mm, x, xs, w, ws, erc, off, _, _ = _case("e4m3", 2, counts, 1040, 256, True, 9)
    rows = sum(counts)
    outs = [cq.grouped_matmul(cfg, mm, x, w, erc, off, x_scales=xs, weight_scales=ws)[:rows] for _ in range(3)]
    codes = [cq.grouped_matmul_quantize(cfg, mm, CODE["e5m2"], x, xs, w, ws, erc, off) for _ in range(3)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert (o == outs[0]).all()
    for c, s in codes[1:]:
        assert (c[:rows] == codes[0][0][:rows]).all() and (s[:rows] == codes[0][1][:rows]).all()
