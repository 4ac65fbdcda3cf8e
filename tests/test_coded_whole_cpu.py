"""That the inputs of test_gpu_coded_whole tell whole products from cut ones (no GPU needed)."""
import pytest
import torch

import experts_ref as ref
import whole_ref as whole


@pytest.mark.parametrize("to", ["e4m3", "e5m2"])
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("I,N,swiglu", [(144, 136, False), (400, 80, False), (272, 160, True)])
def test_cut_products_give_other_codes(kind, to, I, N, swiglu):
    g = torch.Generator()
    g.manual_seed(I)
    counts = [2, 0, 5, 1]
    x, xs, w, ws = whole.inputs(8, counts, I, N, swiglu, kind, g, "cpu")
    _, _, ranges = ref.pack_counts(counts, 2)
    y = whole.sums(x, xs, w, ws, ranges, swiglu)
    assert (y.float().double() == y).all() and (y * 64 == torch.round(y * 64)).all() and y.abs().max() < 2 ** 24
    codes, scales = whole.code(y, to)
    cut, cut_scales = whole.code(whole.sums(x, xs, w, ws, ranges, swiglu, cut=True), to)
    assert (cut & 0x7F == 0).all() and (cut_scales == 0).all()       # nothing is left of them
    assert (scales > 0).all() and (codes != cut).double().mean() > 0.8
