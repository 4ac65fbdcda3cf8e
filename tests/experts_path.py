"""Which kernel a product takes, asked of the library's own rule (csrc/experts_path.h)."""
import ctypes
import os

import combine_quant_amd as cq
from combine_quant_amd import build as B

NAMES = ("stream", "tiles", "small")
TYPES = {"bf16": 0, "f16": 1, "int8": 2, "e4m3": 3, "e5m2": 4, "mx_e4m3": 5, "mx_e5m2": 6}
W4 = {None: 0, "int4": cq.MOE_W4_INT4, "e2m1": cq.MOE_W4_E2M1}


def path(kind, cfg, N, swiglu, w4=None):
    """"stream", "tiles" or "small" for a product of rows of this kind with N weight rows."""
    if not os.path.exists(B.SELFCHECK_LIB):
        raise OSError(f"{B.SELFCHECK_LIB} is missing: build it with combine_quant_amd.build.build()")
    fn = ctypes.CDLL(B.SELFCHECK_LIB).moe_dc_selfcheck_product_path
    fn.argtypes = [ctypes.c_int] * 3 + [ctypes.c_longlong] + [ctypes.c_int] * 2
    fn.restype = ctypes.c_int
    rows = cfg.ep_world_size * cfg.bs * cfg.topk
    return NAMES[fn(TYPES[kind], W4[w4], cfg.moe_expert_num, rows, N, int(swiglu))]
