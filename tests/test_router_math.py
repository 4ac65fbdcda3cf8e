"""The router's exponentials (csrc/gate_math.h), evaluated on the host, against exp in extended
precision: the relative errors their comments state, and the ends of their range."""
import ctypes
import math
import os

import numpy as np
import pytest

from combine_quant_amd import build as B


def _run(which, t):
    if not os.path.exists(B.SELFCHECK_LIB):
        raise OSError(f"{B.SELFCHECK_LIB} is missing: build it with combine_quant_amd.build.build()")
    fn = ctypes.CDLL(B.SELFCHECK_LIB).moe_dc_selfcheck_exp
    fn.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong]
    fn.restype = None
    t = np.ascontiguousarray(t, dtype=np.float64)
    out = np.empty_like(t)
    fn(which, t.ctypes.data, out.ctypes.data, t.size)
    return out


def _error(which, t):
    x = t.astype(np.longdouble)
    want = np.exp2(x) if which == 0 else np.exp(x)
    return float(np.abs(_run(which, t).astype(np.longdouble) / want - 1).max())


# the sums' 2^t: 2^-24.8; the scores' e^x: an ulp, 2^-52
@pytest.mark.parametrize("which,bound,lowest", [(0, 2.0 ** -24.8, -1000.0), (1, 2.0 ** -52, -700.0)])
def test_relative_error(which, bound, lowest):
    g = np.random.default_rng(1)
    for t in (np.linspace(-2, 0, 2_000_001), np.linspace(-41, -40, 500_001),
              lowest * g.random(1_000_000), -np.exp(g.uniform(-60, 0, 500_000))):
        assert _error(which, t) < bound


@pytest.mark.parametrize("which,last", [(0, -1074.0), (1, -745.0)])
def test_ends_of_the_range(which, last):
    out = _run(which, np.array([0.0, -0.0, last, last - 3, last - 100, -1e300, -math.inf, math.nan]))
    assert out[:3].tolist() == [1.0, 1.0, 2.0 ** -1074]
    assert (out[3:7] == 0).all() and math.isnan(out[7])
