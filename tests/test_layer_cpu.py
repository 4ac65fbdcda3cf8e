"""Host-side rules of the experts' layer of a few tokens (no GPU needed)."""
import ctypes
import os
import re

import pytest

import combine_quant_amd as cq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "moe_dc.h")).read()
BASE = 0x100000000
NAMES = ("x", "ids", "weights", "mask", "up", "ups", "down", "downs", "shared", "y")


def _cfg(**kw):
    c = cq.make_config(2, 8, 3, 1024, 2)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _experts(F=144, block=False):
    return cq.make_experts(F, cq.MOE_MM_SCALE_BLOCK if block else cq.MOE_MM_SCALE_NONE)


def _sizes(block, mask):
    each = 1 if block else 2
    n = dict(x=6 * 1024 * 2, ids=48, weights=48, mask={1: 6, 2: 12}.get(mask), up=8 * 288 * 1024 * each,
             ups=8 * 4 * 8 * 4 if block else None, down=8 * 1024 * 144 * each, downs=8 * 8 * 2 * 4 if block else None,
             shared=6 * 1024 * 2, y=6 * 1024 * 2)
    return {k: v for k, v in n.items() if v}


def _apart(sizes):
    at, p = BASE, {}
    for k, n in sizes.items():
        p[k] = at
        at += (n + 4095) // 4096 * 4096
    p["ws"] = at
    return p


def _call(p, cfg=None, experts=None, ws_bytes=None):
    cfg, experts = cfg or _cfg(), _experts() if experts is None else experts
    need = cq.moe_dc_experts_layer_workspace_bytes(cfg, experts) if experts else 0
    P = [None if p.get(k) is None else ctypes.c_void_p(p[k]) for k in NAMES + ("ws",)]
    return cq.load_library().moe_experts_layer(ctypes.byref(cfg), ctypes.byref(experts) if experts else None, *P,
                                               ctypes.c_size_t(need if ws_bytes is None else ws_bytes), None)


def _refused(rc, text, status=cq.MOE_ERR_INVALID_ARG):
    assert rc == status and text in cq.moe_dc_last_error(), (rc, cq.moe_dc_last_error())


def test_descriptor_layout_matches_the_header():
    assert ctypes.sizeof(cq.MoeExperts) == 8
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} moe_experts;", text).group(1)
    assert re.findall(r"(\w+);", body) == [f[0] for f in cq.MoeExperts._fields_]


@pytest.mark.parametrize("cfg,F,block,text", [
    ({}, 0, False, "intermediate"), ({}, 32769, False, "intermediate"), ({}, -8, False, "intermediate"),
    ({}, 12, False, "multiples of 8"), ({}, 24, True, "multiples of 16"), (dict(hidden=1028), 16, False, "multiples"),
    (dict(hidden=1032), 16, True, "multiples"), (dict(bs=0), 16, False, "bs")])
def test_rules(cfg, F, block, text):
    c, e = _cfg(**cfg), _experts(F, block)
    assert cq.moe_dc_experts_layer_workspace_bytes(c, e) == 0
    _refused(_call(_apart(_sizes(block, 0)), c, e, 1 << 30), text)


@pytest.mark.parametrize("scaling", [1, 2, 4, -1])
def test_scaling(scaling):
    _refused(_call(_apart(_sizes(False, 0)), experts=cq.make_experts(144, scaling), ws_bytes=1 << 30), "scaling")


def test_too_many_tokens():
    c = _cfg(bs=33)
    c.expand_rows_capacity = 2 * 33 * 2
    assert cq.moe_dc_experts_layer_workspace_bytes(c, _experts()) == 0
    _refused(_call(_apart(_sizes(False, 0)), c, ws_bytes=1 << 30), "66 tokens", cq.MOE_ERR_UNSUPPORTED)


@pytest.mark.parametrize("name", ["x", "ids", "weights", "up", "down", "y"])
def test_required_pointers(name):
    _refused(_call(dict(_apart(_sizes(False, 0)), **{name: None})), "NULL")


def test_mask_and_scales_pairings():
    p = _apart(_sizes(False, 0))
    _refused(_call(dict(p, mask=BASE)), "mask")
    _refused(_call(p, _cfg(mask_kind=1)), "mask")
    _refused(_call(dict(p, ups=BASE)), "scales")
    _refused(_call(dict(p, downs=BASE)), "scales")
    q = _apart(_sizes(True, 0))
    _refused(_call(dict(q, ups=None), experts=_experts(block=True)), "scales")
    _refused(_call(dict(q, downs=None), experts=_experts(block=True)), "scales")
    _refused(_call(p, experts=False), "NULL")


def test_workspace():
    p = _apart(_sizes(False, 0))
    need = cq.moe_dc_experts_layer_workspace_bytes(_cfg(), _experts())
    assert need >= 6 * 2 * 144 * 2
    _refused(_call(p, ws_bytes=need - 1), "workspace", cq.MOE_ERR_WORKSPACE)
    _refused(_call(dict(p, ws=None)), "workspace", cq.MOE_ERR_WORKSPACE)


@pytest.mark.parametrize("name,off", [("x", 8), ("up", 2), ("down", 8), ("ws", 4), ("ids", 2), ("weights", 1),
                                      ("shared", 1), ("y", 1)])
def test_alignment(name, off):
    p = _apart(_sizes(False, 0))
    p[name] += off
    _refused(_call(p), "aligned")


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("mask", [1, 2])
@pytest.mark.parametrize("out", ["y", "ws"])
@pytest.mark.parametrize("end", ["first", "last"])
def test_overlap(out, block, mask, end):
    cfg, experts, sizes = _cfg(mask_kind=mask), _experts(block=block), _sizes(block, mask)
    need = cq.moe_dc_experts_layer_workspace_bytes(cfg, experts)
    mine = sizes["y"] if out == "y" else need
    for name in sizes:
        if name == out:
            continue
        p = _apart(sizes)
        step = 16 if out == "ws" else 2
        at = p[name] + ((sizes[name] - 1) // step * step if end == "last" else step - mine)
        p[out] = at // step * step
        _refused(_call(p, cfg, experts), "overlap")


def test_binding_refuses_cpu_tensors():
    import torch
    x = torch.zeros((2, 3, 1024), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cq.experts_layer(_cfg(), _experts(), x, torch.zeros((2, 3, 2), dtype=torch.int32), torch.zeros((2, 3, 2)), x, x)
