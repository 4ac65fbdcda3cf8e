"""Host-side rules of the RMS norm (no GPU needed)."""
import ctypes
import os
import re

import pytest

import combine_quant_amd as cq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "moe_dc.h")).read()
BASE = 0x10000000
# 2 x 3 tokens of 1024, mode 3 (8 scales)
SIZES = dict(x=12288, residual=12288, gamma=2048, residual_out=12288, y=12288, codes=6144, scales=192)


def _cfg(mode=3, **kw):
    c = cq.make_config(2, 2, 3, 1024, 1, quant_mode=mode)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _apart():
    at, p = BASE, {}
    for k, n in SIZES.items():
        p[k] = at
        at += (n + 4095) // 4096 * 4096
    return p


def _call(p, cfg=None, norm=None):
    norm = cq.make_norm() if norm is None else norm
    args = [None if p.get(k) is None else ctypes.c_void_p(p[k]) for k in SIZES]
    return cq.load_library().moe_rms_norm(ctypes.byref(cfg or _cfg()),
                                          ctypes.byref(norm) if norm else None, *args, None)


def _refused(rc, text, status=cq.MOE_ERR_INVALID_ARG):
    assert rc == status and text in cq.moe_dc_last_error(), (rc, cq.moe_dc_last_error())


def test_descriptor_layout_matches_the_header():
    assert ctypes.sizeof(cq.MoeNorm) == 8
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} moe_norm;", text).group(1)
    assert re.findall(r"(\w+);", body) == [f[0] for f in cq.MoeNorm._fields_]


@pytest.mark.parametrize("eps", [0.0, -1e-6, float("nan"), float("inf")])
def test_epsilon(eps):
    _refused(_call(_apart(), norm=cq.make_norm(eps)), "epsilon")


def test_description():
    n = cq.make_norm()
    n.reserved = 1
    _refused(_call(_apart(), norm=n), "reserved")
    _refused(cq.load_library().moe_rms_norm(ctypes.byref(_cfg()), None, *[ctypes.c_void_p(v) for v in _apart().values()],
                                            None), "NULL")
    _refused(_call(_apart(), cfg=_cfg(hidden=1000)), "hidden")


@pytest.mark.parametrize("kw", [
    dict(mode=1, scales_kind=cq.MOE_SCALES_SCALAR), dict(mode=2, scales_kind=cq.MOE_SCALES_SHARED),
    dict(mode=3, scales_kind=cq.MOE_SCALES_PER_EXPERT), dict(mode=4, out_dtype=cq.MOE_DTYPE_E2M1)])
def test_unsupported(kw):
    _refused(_call(_apart(), cfg=_cfg(**kw)), "", cq.MOE_ERR_UNSUPPORTED)


@pytest.mark.parametrize("mode,missing", [(3, "x"), (3, "gamma"), (3, "codes"), (3, "scales"), (3, "residual")])
def test_required_pointers(mode, missing):
    _refused(_call(dict(_apart(), **{missing: None}), cfg=_cfg(mode)), "")


def test_mode_0():
    p = _apart()
    _refused(_call(p, cfg=_cfg(0)), "iff")
    _refused(_call(dict(p, codes=None, scales=None, y=None), cfg=_cfg(0)), "y is required")


@pytest.mark.parametrize("name", ["x", "residual", "gamma", "residual_out", "y", "scales"])
def test_alignment(name):
    p = _apart()
    p[name] += 1
    _refused(_call(p), "aligned")


@pytest.mark.parametrize("out", ["residual_out", "y", "codes", "scales"])
@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("end", ["first", "last"])
def test_overlap(out, name, end):
    if out == name:
        return
    p = _apart()
    p[out] = p[name] + (SIZES[name] - 4 if end == "last" else 4 - SIZES[out])
    _refused(_call(p), "overlap")


@pytest.mark.parametrize("out,name", [("codes", "x"), ("scales", "residual"), ("y", "gamma"), ("y", "residual_out")])
def test_in_place_of_the_wrong_tensor(out, name):
    p = _apart()
    p[out] = p[name]
    _refused(_call(p), "overlap")


def test_binding_refuses_cpu_tensors():
    import torch
    with pytest.raises(ValueError):
        cq.rms_norm(_cfg(), cq.make_norm(), torch.zeros((2, 3, 1024), dtype=torch.bfloat16),
                    torch.zeros(1024, dtype=torch.bfloat16))
