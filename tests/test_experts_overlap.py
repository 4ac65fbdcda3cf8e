"""Outputs of the router and the products that share memory with what the same call reads are
refused (host only: the refusal comes before any device work)."""
import ctypes

import pytest

import combine_quant_amd as cq

BASE = 0x10000000


def _refused(rc):
    assert rc == cq.MOE_ERR_INVALID_ARG and "overlap" in cq.moe_dc_last_error()


def _cfg():
    return cq.make_config(2, 8, 16, 1024, 2)                         # 64 rows


# bytes: x 64 * 128 * 2, weights 8 * 96 * 128 * 2, counts 2 * 8 * 4, offsets 3 * 8, out 64 * 96 * 2
TOKENS = dict(x=16384, w=196608, erc=64, off=24, out=12288)


def _product(cfg, mm, p, xs=None, ws=None):
    P = {k: None if v is None else ctypes.c_void_p(v) for k, v in dict(p, xs=xs, ws=ws).items()}
    return cq.load_library().moe_grouped_matmul(
        ctypes.byref(cfg), ctypes.byref(mm), P["x"], P["xs"], P["w"], P["ws"], P["erc"], P["off"],
        P["out"], None)


def _apart(sizes):
    at, p = BASE, {}
    for k, n in sizes.items():
        p[k] = at
        at += (n + 4095) // 4096 * 4096
    return p


@pytest.mark.parametrize("name", ["x", "w", "erc", "off"])
@pytest.mark.parametrize("end", ["first", "last"])
def test_product_output(name, end):
    p = _apart(TOKENS)
    p["out"] = p[name] + (TOKENS[name] - 8 if end == "last" else 16 - TOKENS["out"])
    _refused(_product(_cfg(), cq.make_matmul(128, 96), p))


def test_product_in_place():
    p = _apart(TOKENS)
    p["out"] = p["x"]
    _refused(_product(_cfg(), cq.make_matmul(128, 128), p))


def test_rows_beyond_any_batch_do_not_count():
    """A capacity above W * BS * K does not make buffers that hold the batch's rows overlap: the call
    gets past the checks (and, without a GPU, no further)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("host rule; the pointers are not a GPU's")
    cfg = _cfg()
    cfg.expand_rows_capacity = (1 << 31) - 1
    assert _product(cfg, cq.make_matmul(128, 96), _apart(TOKENS)) == cq.MOE_ERR_DEVICE


@pytest.mark.parametrize("which", ["xs", "ws"])
@pytest.mark.parametrize("kind", ["row", "mx"])
def test_product_output_and_scales(which, kind):
    mx = kind == "mx"
    mm = cq.make_matmul(128, 96, x_dtype=cq.MOE_DTYPE_E4M3,
                        scaling=cq.MOE_MM_SCALE_MX if mx else cq.MOE_MM_SCALE_ROW)
    xs, ws = BASE + (1 << 24), BASE + (1 << 25)
    size = {"xs": 64 * 4, "ws": 8 * 96 * 4}[which]                   # the same for both
    p = _apart(TOKENS)
    p["out"] = {"xs": xs, "ws": ws}[which] + size - 4
    _refused(_product(_cfg(), mm, p, xs, ws))


@pytest.mark.parametrize("which,size", [("x", 16384), ("w", 8 * 96 * 64), ("ws", 8 * 96 * 2 * 2),
                                        ("erc", 64), ("off", 24)])
def test_4bit_product_output(which, size):
    p = _apart(dict(TOKENS, ws=4096))
    p["out"] = p[which] + size - 8
    P = {k: ctypes.c_void_p(v) for k, v in p.items()}
    cfg, mm = _cfg(), cq.make_matmul(128, 96, weight_dtype=cq.MOE_W4_INT4, group_size=64)
    _refused(cq.load_library().moe_grouped_matmul_w4(
        ctypes.byref(cfg), ctypes.byref(mm), P["x"], P["w"], P["ws"], P["erc"], P["off"], P["out"], None))


@pytest.mark.parametrize("a,b,size", [("ids", "logits", 32 * 8 * 4), ("weights", "logits", 32 * 8 * 4),
                                      ("ids", "bias", 32), ("weights", "bias", 32),
                                      ("ids", "weights", 32 * 2 * 4)])
def test_router_outputs(a, b, size):
    p = _apart(dict(logits=1024, bias=32, ids=256, weights=256))
    p[a] = p[b] + size - 4
    P = {k: ctypes.c_void_p(v) for k, v in p.items()}
    cfg, gate = _cfg(), cq.make_gate()
    _refused(cq.load_library().moe_gate_topk(
        ctypes.byref(cfg), ctypes.byref(gate), P["logits"], P["bias"], P["ids"], P["weights"], None))
