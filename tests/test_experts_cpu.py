"""Host-side rules of the router and the experts' products (no GPU needed): descriptor layouts,
enum values, and every refusal, which happens before any device work."""
import ctypes
import os
import re

import pytest

import combine_quant_amd as cq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "moe_dc.h")).read()
P = ctypes.c_void_p(0x1000)


def test_descriptor_layouts_match_the_header():
    assert ctypes.sizeof(cq.MoeMatmul) == 32 and ctypes.sizeof(cq.MoeGate) == 24
    for cls, name in ((cq.MoeMatmul, "moe_matmul"), (cq.MoeGate, "moe_gate")):
        text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text).group(1)
        assert re.findall(r"(\w+);", body) == [f[0] for f in cls._fields_]


@pytest.mark.parametrize("name", [
    "MOE_MM_SCALE_NONE", "MOE_MM_SCALE_ROW", "MOE_MM_SCALE_MX", "MOE_ACT_NONE", "MOE_ACT_SWIGLU",
    "MOE_W4_INT4", "MOE_W4_E2M1", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID"])
def test_enum_values_match_the_binding(name):
    m = re.search(r"\b" + name + r"\s*=\s*(\d+)", HEADER)
    assert m and int(m.group(1)) == getattr(cq, name)


def _cfg(**kw):
    c = cq.make_config(2, 8, 16, 1024, 2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _mm(lib, cfg, mm, x=P, xs=None, w=P, ws=None, erc=P, off=P, out=P):
    return lib.moe_grouped_matmul(ctypes.byref(cfg), ctypes.byref(mm) if mm else None, x, xs, w,
                                  ws, erc, off, out, None)


def _w4(lib, cfg, mm, x=P, w=P, ws=P, erc=P, off=P, out=P):
    return lib.moe_grouped_matmul_w4(ctypes.byref(cfg), ctypes.byref(mm), x, w, ws, erc, off,
                                     out, None)


def _gate(lib, cfg, gate, logits=P, ids=P, weights=P):
    return lib.moe_gate_topk(ctypes.byref(cfg), ctypes.byref(gate) if gate else None, logits,
                             None, ids, weights, None)


ROW, MX = cq.MOE_MM_SCALE_ROW, cq.MOE_MM_SCALE_MX
I8, E4, E5 = cq.MOE_DTYPE_INT8, cq.MOE_DTYPE_E4M3, cq.MOE_DTYPE_E5M2


@pytest.mark.parametrize("args,kw,text", [
    ((0, 64), {}, "in_features"), ((65537, 64), {}, "in_features"), ((-8, 64), {}, "in_features"),
    ((64, 0), {}, "out_features"), ((64, 65537), {}, "out_features"),
    ((64, 63), dict(activation=1), "even"), ((64, 64), dict(activation=2), "activation"),
    ((64, 64), dict(activation=-1), "activation"),
    ((1020, 64), {}, "multiple of 8"), ((1032, 64), dict(x_dtype=I8, scaling=ROW), "multiple of 16"),
    ((1024 + 32, 64), dict(x_dtype=E4, scaling=MX), "multiple of 128"),
    ((64, 64), dict(scaling=ROW), "scal"), ((64, 64), dict(scaling=3), "scaling"),
    ((64, 64), dict(scaling=-1), "scaling"), ((64, 64), dict(x_dtype=I8), "scaling"),
    ((128, 64), dict(x_dtype=I8, scaling=MX), "scaling"), ((64, 64), dict(x_dtype=E4), "scaling"),
    ((64, 64), dict(x_dtype=7), "x_dtype"), ((64, 64), dict(weight_dtype=1), "weight_dtype"),
    ((64, 64), dict(group_size=32), "group_size"),
])
def test_product_rules(args, kw, text):
    lib = cq.load_library()
    rc = _mm(lib, _cfg(), cq.make_matmul(*args, **kw))
    assert rc == cq.MOE_ERR_INVALID_ARG and text in cq.moe_dc_last_error()


def test_product_pointer_rules():
    lib = cq.load_library()
    c = _cfg()
    tok, row, mx = (cq.make_matmul(128, 64), cq.make_matmul(128, 64, x_dtype=I8, scaling=ROW),
                    cq.make_matmul(128, 64, x_dtype=E5, scaling=MX))
    for kw in (dict(x=None), dict(w=None), dict(erc=None), dict(off=None), dict(out=None)):
        assert _mm(lib, c, tok, **kw) == cq.MOE_ERR_INVALID_ARG
        assert "NULL" in cq.moe_dc_last_error()
    for kw in (dict(x=ctypes.c_void_p(0x1008)), dict(w=ctypes.c_void_p(0x1008))):
        assert _mm(lib, c, tok, **kw) == cq.MOE_ERR_INVALID_ARG
        assert "aligned" in cq.moe_dc_last_error()
    for mm, kw in ((tok, dict(xs=P)), (tok, dict(ws=P)), (row, {}), (row, dict(xs=P)),
                   (mx, dict(ws=P)), (mx, dict(xs=P))):
        assert _mm(lib, c, mm, **kw) == cq.MOE_ERR_INVALID_ARG
        assert "scales" in cq.moe_dc_last_error()
    assert _mm(lib, c, None) == cq.MOE_ERR_INVALID_ARG
    e2m1 = cq.make_matmul(128, 64, x_dtype=cq.MOE_DTYPE_E2M1, scaling=MX)
    assert _mm(lib, c, e2m1, xs=P, ws=P) == cq.MOE_ERR_UNSUPPORTED
    bad = cq.make_matmul(128, 64)
    bad.reserved = 1
    assert _mm(lib, c, bad) == cq.MOE_ERR_INVALID_ARG
    assert _mm(lib, _cfg(bs=513), tok) == cq.MOE_ERR_INVALID_ARG      # the config's own rules


@pytest.mark.parametrize("args,kw,text", [
    ((128, 64), dict(weight_dtype=0, group_size=32), "weight_dtype"),
    ((128, 64), dict(weight_dtype=3, group_size=32), "weight_dtype"),
    ((128, 64), dict(weight_dtype=1, group_size=16), "group_size"),
    ((128, 64), dict(weight_dtype=1, group_size=0), "group_size"),
    ((128, 64), dict(weight_dtype=2, group_size=64), "E2M1"),
    ((96, 64), dict(weight_dtype=1, group_size=64), "multiple"),
    ((48, 64), dict(weight_dtype=2, group_size=32), "multiple"),
    ((128, 64), dict(weight_dtype=1, group_size=64, x_dtype=I8), "token"),
    ((128, 64), dict(weight_dtype=1, group_size=64, scaling=ROW), "token"),
    ((128, 63), dict(weight_dtype=1, group_size=64, activation=1), "even"),
])
def test_4bit_product_rules(args, kw, text):
    lib = cq.load_library()
    rc = _w4(lib, _cfg(), cq.make_matmul(*args, **kw))
    assert rc == cq.MOE_ERR_INVALID_ARG and text in cq.moe_dc_last_error()


def test_4bit_product_pointer_rules():
    lib = cq.load_library()
    mm = cq.make_matmul(128, 64, weight_dtype=cq.MOE_W4_INT4, group_size=64)
    for kw in (dict(x=None), dict(w=None), dict(ws=None), dict(erc=None), dict(off=None),
               dict(out=None), dict(w=ctypes.c_void_p(0x1004))):
        assert _w4(lib, _cfg(), mm, **kw) == cq.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("cfg,kw,status", [
    ({}, dict(score=2), cq.MOE_ERR_INVALID_ARG), ({}, dict(score=-1), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=0), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=3), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=2, group_keep=3), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=2, group_keep=0), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=2, group_top=3), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=8, group_top=2, group_keep=8), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(group_count=8), cq.MOE_ERR_INVALID_ARG),            # topk 2, one id kept
    ({}, dict(factor=float("nan")), cq.MOE_ERR_INVALID_ARG),
    ({}, dict(factor=float("inf")), cq.MOE_ERR_INVALID_ARG),
    (dict(zero_expert_num=2041), {}, cq.MOE_ERR_UNSUPPORTED),
    (dict(topk=17), {}, cq.MOE_ERR_INVALID_ARG),
])
def test_router_rules(cfg, kw, status):
    lib = cq.load_library()
    assert _gate(lib, _cfg(**cfg), cq.make_gate(**kw)) == status
    assert cq.moe_dc_last_error() != ""


def test_router_pointer_rules():
    lib = cq.load_library()
    for kw in (dict(logits=None), dict(ids=None), dict(weights=None)):
        assert _gate(lib, _cfg(), cq.make_gate(), **kw) == cq.MOE_ERR_INVALID_ARG
    assert _gate(lib, _cfg(), None) == cq.MOE_ERR_INVALID_ARG
    g = cq.make_gate()
    g.renormalize = 2
    assert _gate(lib, _cfg(), g) == cq.MOE_ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors():
    import torch
    c = _cfg()
    x = torch.zeros((64, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cq.grouped_matmul(c, cq.make_matmul(64, 64), x, x, x, x)
    with pytest.raises(ValueError):
        cq.gate_topk(c, cq.make_gate(), torch.zeros((2, 16, 8)))
