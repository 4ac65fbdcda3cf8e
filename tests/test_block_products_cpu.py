"""Host-side rules of the block-scaled products (no GPU needed)."""
import ctypes

import pytest

import combine_quant_amd as cq

BASE = 0x10000000
E4, E5, BLOCK = cq.MOE_DTYPE_E4M3, cq.MOE_DTYPE_E5M2, cq.MOE_MM_SCALE_BLOCK
# 64 rows, I = 144 (two groups), N = 160 (two rows of blocks), 8 experts
SIZES = dict(x=64 * 144, xs=64 * 2 * 4, w=8 * 160 * 144, ws=8 * 2 * 2 * 4, erc=64, off=24,
             out=64 * 160 * 2)


def _cfg(**kw):
    c = cq.make_config(2, 8, 16, 1024, 2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _mm(I=144, N=160, **kw):
    return cq.make_matmul(I, N, **dict(dict(x_dtype=E4, scaling=BLOCK), **kw))


def _apart(sizes):
    at, p = BASE, {}
    for k, n in sizes.items():
        p[k] = at
        at += (n + 4095) // 4096 * 4096
    return p


def _tokens(mm, p, cfg=None):
    P = {k: None if v is None else ctypes.c_void_p(v) for k, v in p.items()}
    return cq.load_library().moe_grouped_matmul(
        ctypes.byref(cfg or _cfg()), ctypes.byref(mm) if mm else None, P["x"], P["xs"], P["w"],
        P["ws"], P["erc"], P["off"], P["out"], None)


def _codes(mm, p, to=E4, cfg=None):
    P = {k: None if v is None else ctypes.c_void_p(v) for k, v in p.items()}
    return cq.load_library().moe_grouped_matmul_quantize(
        ctypes.byref(cfg or _cfg()), ctypes.byref(mm) if mm else None, to, P["x"], P["xs"], P["w"],
        P["ws"], P["erc"], P["off"], P["out"], P["os"], None)


CODED = dict(SIZES, out=64 * 160, os=64 * 2 * 4)


def _refused(rc, text):
    assert rc == cq.MOE_ERR_INVALID_ARG and text in cq.moe_dc_last_error(), cq.moe_dc_last_error()


@pytest.mark.parametrize("kw,text", [
    (dict(x_dtype=0), "scales"), (dict(x_dtype=cq.MOE_DTYPE_INT8), "scaling"), (dict(I=136), "multiple of 16"),
    (dict(scaling=4), "scaling"), (dict(N=161, activation=1), "even"), (dict(group_size=32), "group_size"),
])
def test_rules(kw, text):
    _refused(_tokens(_mm(**kw), _apart(SIZES)), text)


@pytest.mark.parametrize("kw,text", [
    (dict(scaling=cq.MOE_MM_SCALE_ROW), "BLOCK"), (dict(x_dtype=0, scaling=0), "BLOCK"),
    (dict(x_dtype=cq.MOE_DTYPE_INT8), "scaling"), (dict(I=136), "multiple of 16"),
    (dict(N=0), "out_features"), (dict(weight_dtype=1), "weight_dtype"),
])
def test_coded_rules(kw, text):
    _refused(_codes(_mm(**kw), _apart(CODED)), text)


@pytest.mark.parametrize("to", [0, 1, 4, -1, 9])
def test_coded_types(to):
    _refused(_codes(_mm(), _apart(CODED), to), "out_dtype")


def test_required_pointers():
    for name in SIZES:
        _refused(_tokens(_mm(), dict(_apart(SIZES), **{name: None})), "")
    for name in CODED:
        _refused(_codes(_mm(), dict(_apart(CODED), **{name: None})), "")
    _refused(_codes(None, _apart(CODED)), "NULL")
    _refused(_codes(_mm(), _apart(CODED), cfg=_cfg(bs=513)), "bs")


@pytest.mark.parametrize("name,off", [("x", 8), ("w", 4), ("xs", 2), ("ws", 1), ("os", 2)])
def test_alignment(name, off):
    p = _apart(CODED)
    p[name] += off
    _refused(_codes(_mm(), p), "aligned")


@pytest.mark.parametrize("out", ["out", "os"])
@pytest.mark.parametrize("name", ["x", "xs", "w", "ws", "erc", "off"])
@pytest.mark.parametrize("end", ["first", "last"])
def test_coded_outputs_apart_from_inputs(out, name, end):
    p = _apart(CODED)
    p[out] = p[name] + (CODED[name] - 4 if end == "last" else 4 - CODED[out])
    _refused(_codes(_mm(), p), "overlap")


def test_coded_outputs_apart():
    p = _apart(CODED)
    p["os"] = p["out"] + CODED["out"] - 4
    _refused(_codes(_mm(), p), "overlap")


@pytest.mark.parametrize("name", ["xs", "ws"])
def test_output_and_scales(name):
    p = _apart(SIZES)
    p["out"] = p[name] + SIZES[name] - 4
    _refused(_tokens(_mm(), p), "overlap")
    # with SwiGLU the gate and the up rows have blocks of their own: 80 rows are one row each
    p["out"] = p["ws"] + 8 * 2 * 2 * 4 - 4
    _refused(_tokens(_mm(activation=cq.MOE_ACT_SWIGLU), p), "overlap")


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros((64, 144), dtype=torch.uint8)
    s = torch.zeros((64, 2))
    with pytest.raises(ValueError):
        cq.grouped_matmul_quantize(_cfg(), _mm(), E4, x, s, x, s, s, s)


@pytest.mark.parametrize("E,rows,N,swiglu,coded,want", [
    # large tiles of 224 rows x 256 columns (SwiGLU 128 of each half): from 192 of them on
    (64, 2048, 768, False, 0, 1), (64, 2048, 512, False, 0, 3), (8, 4096, 2048, True, 0, 1), (8, 4096, 1792, True, 0, 3),
    # streaming: up to 32 rows an expert and fewer than 96 thin tiles of 64 rows x 128 columns
    (8, 256, 11 * 128, False, 0, 0), (8, 256, 12 * 128, False, 0, 3), (8, 264, 128, False, 0, 3),
    (8, 64, 11 * 128, True, 0, 0), (8, 64, 12 * 128, True, 0, 3), (8, 4, 1024, False, 0, 0),
    # coded results: never streamed, and gate and up in large tiles
    (8, 64, 128, False, 2, 3), (8, 64, 128, True, 3, 1), (64, 2048, 768, False, 2, 1),
])
@pytest.mark.parametrize("kind", [7, 8])
def test_which_kernel(kind, E, rows, N, swiglu, coded, want):
    import ctypes
    from combine_quant_amd import build as B
    fn = ctypes.CDLL(B.SELFCHECK_LIB).moe_dc_selfcheck_coded_product_path
    fn.argtypes = [ctypes.c_int] * 2 + [ctypes.c_longlong] + [ctypes.c_int] * 3
    fn.restype = ctypes.c_int
    assert fn(kind, E, rows, N, int(swiglu), coded) == want
