"""The rule that chooses a product's kernel (host only)."""
import pytest

import combine_quant_amd as cq
from experts_path import path


@pytest.mark.parametrize("kind,E,rows,N,swiglu,want", [
    # 56 tiles of 256 (MX 192) rows x 256 columns (SwiGLU: 128 of each half)
    ("bf16", 8, 16, 7 * 256, False, "tiles"), ("bf16", 8, 16, 6 * 256, False, "stream"),
    ("int8", 8, 16, 7 * 256, True, "tiles"), ("int8", 8, 16, 6 * 256, True, "stream"),
    ("f16", 8, 2048, 7 * 256, False, "tiles"), ("f16", 8, 2064, 3 * 256, False, "stream"),
    ("mx_e4m3", 8, 1536, 6 * 256, False, "stream"), ("mx_e4m3", 8, 1552, 4 * 256, False, "tiles"),
    ("e4m3", 256, 16, 3 * 256, False, "stream"), ("e4m3", 256, 16, 4 * 256, False, "tiles"),
])
def test_product_path(kind, E, rows, N, swiglu, want):
    cfg = cq.make_config(2, E, rows // 16, 1024, 8)
    assert path(kind, cfg, N, swiglu) == want


@pytest.mark.parametrize("E,rows,N,swiglu,want", [
    (8, 16, 18 * 128, False, "small"), (8, 16, 17 * 128, False, "stream"),
    (8, 16, 9 * 256, True, "small"), (8, 16, 8 * 256, False, "stream"),
    (8, 256, 18 * 128, False, "small"), (8, 272, 18 * 128, False, "stream"), (8, 272, 20 * 128, False, "tiles"),
    (8, 1024, 10 * 256, False, "tiles"), (8, 1024, 9 * 256, False, "stream"),
])
@pytest.mark.parametrize("w4", ["int4", "e2m1"])
def test_4bit_product_path(w4, E, rows, N, swiglu, want):
    cfg = cq.make_config(2, E, rows // 16, 1024, 8)
    assert path("bf16", cfg, N, swiglu, w4) == want
