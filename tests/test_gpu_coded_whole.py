"""Coded results of tiles of up to 64 rows come of whole products: inputs of which the fp8 matrix
instructions alone would leave nothing, and codes and scales to the bit (whole_ref)."""
import pytest
import torch

import block_ref as blk
import combine_quant_amd as cq
import experts_ref as ref
import whole_ref as whole
from test_gpu_block_products import CODE, _config, _desc

pytestmark = pytest.mark.gpu

DEV = "cuda"
THIN, LARGE = 3, 1
FEW = [5, 0, 33, 64, 16, 48]                                # every height of a thin tile
MANY = [(5 * e) % 4 for e in range(251)] + [64, 17, 40, 50, 1]        # 256 experts


@pytest.mark.parametrize("kind,to", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("counts,I,N,swiglu,path", [
    (FEW, 144, 136, False, THIN), (FEW, 656, 300, False, THIN), (FEW, 272, 320, True, LARGE),
    (MANY, 144, 200, False, LARGE), (MANY, 528, 144, True, LARGE)])
def test_codes_of_whole_products(kind, to, counts, I, N, swiglu, path):
    g = torch.Generator(device=DEV)
    g.manual_seed(I + N)
    cfg = _config(2, counts)
    assert whole.path(kind, cfg, N, swiglu, to) == path
    x, xs, w, ws = whole.inputs(cfg.expand_rows_capacity, counts, I, N, swiglu, kind, g, DEV)
    erc, off, ranges = ref.pack_counts(counts, 2)
    codes, scales = cq.grouped_matmul_quantize(cfg, _desc(kind, I, N, swiglu), CODE[to], x, xs, w, ws, erc.to(DEV),
                                               off.to(DEV))
    torch.cuda.synchronize()
    rows = sum(counts)
    y = whole.sums(x.cpu(), xs.cpu(), w.cpu(), ws.cpu(), ranges, swiglu)
    want, ws_ = whole.code(y, to)
    assert want.shape[1] == (N // 2 if swiglu else N) and ws_.shape[1] == blk.groups(want.shape[1])
    got = codes[:rows].cpu()
    # the sign of a zero does not matter
    differ = (got != want) & ~((got & 0x7F == 0) & (want & 0x7F == 0))
    assert not differ.any(), (int(differ.sum()), differ.numel())
    assert (scales[:rows].cpu() == ws_).all()
