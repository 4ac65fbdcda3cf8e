"""Workspaces that a call or a plan allocates itself, used on a stream that is not the current one:
memory that the current stream allocates and fills meanwhile must not be theirs."""
import pytest
import torch

import combine_quant_amd as cq
from test_gpu_layer import Case

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _layer():
    """(one call on a stream, a plan, result)"""
    c = Case(2, 16, 16, 4, 1024, 272, seed=21)
    n = cq.moe_dc_experts_layer_workspace_bytes(c.cfg, c.experts)
    args = (c.cfg, c.experts, c.x, c.ids, c.weight, c.up, c.down)
    return (lambda y, s: cq.experts_layer(*args, y=y, stream=s), lambda y: cq.prepare_experts_layer(*args, y=y)[0], n)


def _scatter():
    W, E, BS, H, K = 2, 16, 64, 1024, 4
    g = torch.Generator(device=DEV)
    g.manual_seed(22)
    cfg = cq.make_config(W, E, BS, H, K)
    ids = torch.rand((W, BS, E), generator=g, device=DEV).topk(K, 2).indices.int()
    x = torch.randn((W, BS, H), generator=g, device=DEV).bfloat16()
    w = torch.rand((W, BS, K), generator=g, device=DEV)
    d = cq.dispatch(cfg, x, ids)
    args = (cfg, d["expand_x"], d["assist_info"], d["recv_offsets"], ids, w)
    n = cq.moe_dc_combine_scatter_workspace_bytes(cfg)
    return (lambda y, s: cq.combine_scatter(*args, y=y, stream=s),
            lambda y: cq.prepare_combine_scatter(*args, y=y)[0], n)


@pytest.mark.parametrize("planned", [False, True])
@pytest.mark.parametrize("make", [_layer, _scatter])
def test_current_stream_goes_on_allocating(make, planned):
    call, plan, n = make()
    want = call(None, None)
    y = torch.zeros_like(want)
    big = torch.randn((4096, 4096), device=DEV)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        y.zero_()
        launch = plan(y) if planned else None
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(8):
                big @ big                                   # the call below waits behind these
        if planned:
            launch(s)
            del launch
        else:
            call(y, s)
        held = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(16)]
        assert not s.query()                                # the call had not run when they were filled
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del held


@pytest.mark.parametrize("make", [_layer, _scatter])
def test_captured_plan_with_its_own_workspace(make):
    call, plan, n = make()
    want = call(None, None)
    y = torch.zeros_like(want)
    launch, s, graph = plan(y), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        launch()
    for _ in range(4):
        y.zero_()
        graph.replay()
        held = [torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        y.zero_()
        launch()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
        del held
