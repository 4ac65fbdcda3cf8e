"""Norm, router, dispatch, coded products and combine run together, and the layer of a few tokens in
their place: on a side stream without synchronising, from plans and captured in graphs.  Every stage
is compared with the plain 64-bit form of its actual inputs."""
import math

import pytest
import torch

import block_ref as blk
import combine_quant_amd as cq
import experts_ref as ref
import layer_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BLOCK, SWIGLU, E4 = cq.MOE_MM_SCALE_BLOCK, cq.MOE_ACT_SWIGLU, cq.MOE_DTYPE_E4M3


def _weights(E, parts, n, k, g):
    """E4M3 weights [E][parts * n][k] with their blocks' scales."""
    w = torch.empty((E, parts, n, k), dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty((E, parts, blk.groups(n), blk.groups(k)), device=DEV)
    for e in range(E):
        for p in range(parts):
            v = torch.randn((n, k), generator=g, device=DEV) / math.sqrt(k)
            pad = torch.nn.functional.pad(v.abs(), (0, -k % 128, 0, -n % 128))
            s[e, p] = pad.view(blk.groups(n), 128, blk.groups(k), 128).amax((1, 3)) / 448
            wide = s[e, p].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
            w[e, p] = (v / wide).clamp(-448, 448).to(torch.float8_e4m3fn)
    return w.view(E, parts * n, k), s.view(E, parts * blk.groups(n), blk.groups(k))


class Layer:
    """x, residual -> norm -> router and shared expert; experts by the packed path (`packed`) or by
    the layer of a few tokens -> y."""

    def __init__(self, W, E, BS, H, F, K, packed, f16=False, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        token = torch.float16 if f16 else torch.bfloat16
        self.packed, self.H, self.F, self.g = packed, H, F, g
        kind = dict(token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16, out_dtype=E4)
        self.cfg = cq.make_config(W, E, BS, H, K, 3, **kind)
        self.scfg = cq.make_config(W, W, BS, H, 1, 3, **kind)      # the shared expert: one per rank
        self.x = torch.randn((W, BS, H), generator=g, device=DEV).to(token)
        self.residual = (torch.randn((W, BS, H), generator=g, device=DEV) * 3).to(token)
        self.gamma = (0.5 + torch.rand((H,), generator=g, device=DEV)).to(token)
        self.wg = torch.randn((H, E), generator=g, device=DEV) / math.sqrt(H)
        self.gate = cq.make_gate(cq.MOE_SCORE_SIGMOID, renormalize=True, factor=2.5)
        self.up, self.ups = _weights(E, 2, F, H, g)
        self.down, self.downs = _weights(E, 1, H, F, g)
        up, ups = _weights(1, 2, F, H, g)
        down, downs = _weights(1, 1, H, F, g)
        self.sup, self.sups, self.sdown, self.sdowns = (t.expand(W, -1, -1).contiguous()
                                                        for t in (up, ups, down, downs))
        self.mm1 = cq.make_matmul(H, 2 * F, x_dtype=E4, scaling=BLOCK, activation=SWIGLU)
        self.mm2 = cq.make_matmul(F, H, x_dtype=E4, scaling=BLOCK)
        # rank r's tokens are the rows of its own copy of the shared expert
        self.erc = torch.tensor([[BS if s >= r else 0 for s in range(W)] for r in range(W)],
                                dtype=torch.int32, device=DEV)
        self.off = torch.arange(W + 1, dtype=torch.int64, device=DEV) * BS

    def new_inputs(self):
        self.x.copy_(torch.randn(self.x.shape, generator=self.g, device=DEV))
        self.residual.copy_(torch.randn(self.x.shape, generator=self.g, device=DEV) * 3)

    def run(self, stream=None):
        cfg, T = self.cfg, self.x.shape[0] * self.x.shape[1]
        n = cq.rms_norm(cfg, cq.make_norm(), self.x, self.gamma, residual=self.residual, stream=stream)
        sc, ss = cq.grouped_matmul_quantize(
            self.scfg, self.mm1, E4, n["codes"].view(T, self.H), n["dynamic_scales"].view(T, -1), self.sup,
            self.sups, self.erc, self.off, stream=stream)
        shared = cq.grouped_matmul(self.scfg, self.mm2, sc, self.sdown, self.erc, self.off, x_scales=ss,
                                   weight_scales=self.sdowns, stream=stream).view(self.x.shape)
        logits = n["y"].float() @ self.wg
        ids, w = cq.gate_topk(cfg, self.gate, logits, stream=stream)
        got = dict(n, sc=sc, ss=ss, shared=shared, ids=ids, w=w)
        if not self.packed:
            got["out"] = cq.experts_layer(
                cfg, cq.make_experts(self.F, BLOCK), n["y"], ids, w, self.up, self.down, up_scales=self.ups,
                down_scales=self.downs, shared_x=shared, stream=stream)
            return got
        d = cq.dispatch(cfg, n["y"], ids, stream=stream)
        h, hs = cq.grouped_matmul_quantize(cfg, self.mm1, E4, d["expand_x"], d["dynamic_scales"], self.up,
                                           self.ups, d["ep_recv_count"], d["recv_offsets"], stream=stream)
        o = cq.grouped_matmul(cfg, self.mm2, h, self.down, d["ep_recv_count"], d["recv_offsets"],
                              x_scales=hs, weight_scales=self.downs, stream=stream)
        out = cq.combine_scatter(cfg, o, d["assist_info"], d["recv_offsets"], ids, w, shared_x=shared,
                                 stream=stream)
        return dict(got, d=d, h=h, hs=hs, o=o, out=out)

    def check(self, r):
        token, T = self.x.dtype, self.x.shape[0] * self.x.shape[1]
        s = self.x.double() + self.residual.double()
        y = s / torch.sqrt((s * s).mean(2, keepdim=True) + 1e-6) * self.gamma.double()
        half = ref.HALF_STEP[token]
        assert ((r["y"].double() - y).abs() <= (2.0 ** -18 + half * 1.001) * y.abs() + 2.0 ** -25).all()
        f8 = torch.float8_e4m3fn
        blk.check_codes(r["codes"].view(T, self.H).view(f8), r["dynamic_scales"].view(T, -1), y.view(T, -1),
                        2.0 ** -18 * y.view(T, -1).abs(), "e4m3", T)
        W, BS = self.x.shape[:2]
        ranges = [(i * BS, (i + 1) * BS) for i in range(W)]
        v, e = blk.product(r["codes"].view(T, -1).view(f8), r["dynamic_scales"].view(T, -1), self.sup, self.sups, ranges, True)
        blk.check_codes(r["sc"].view(f8), r["ss"], v, e, "e4m3", T)
        v, e = blk.product(r["sc"].view(f8), r["ss"], self.sdown, self.sdowns, ranges, False)
        ref.check(r["shared"].view(T, -1), v, e, T)
        if not self.packed:
            v, e = layer_ref.layer(self.cfg, r["y"].double().view(T, -1), r["ids"], r["w"],
                                   blk.weights_f64(self.up, self.ups, 2), blk.weights_f64(self.down, self.downs, 1),
                                   shared=r["shared"])
            ref.check(r["out"].view(T, -1), v, e, T)
            return
        d, rows = r["d"], T * self.cfg.topk
        per = torch.bincount(r["ids"].flatten().long(), minlength=self.cfg.moe_expert_num)
        ends = per.cumsum(0).tolist()
        ranges = list(zip([0] + ends[:-1], ends))
        v, e = blk.product(d["expand_x"][:rows].view(f8), d["dynamic_scales"][:rows], self.up, self.ups, ranges, True)
        blk.check_codes(r["h"].view(f8), r["hs"], v, e, "e4m3", rows)
        v, e = blk.product(r["h"][:rows].view(f8), r["hs"][:rows], self.down, self.downs, ranges, False)
        ref.check(r["o"], v, e, rows)
        a = d["assist_info"][:rows].long()
        flat = (a[:, 0] * BS + a[:, 1])
        weight = r["w"].view(T, -1)[flat, a[:, 2]].double()
        part = r["o"][:rows].double() * weight[:, None]
        want = r["shared"].double().view(T, -1).index_add(0, flat, part)
        mag = r["shared"].double().view(T, -1).abs().index_add(0, flat, part.abs())
        ref.check(r["out"].view(T, -1), want, (self.cfg.topk + 2) * ref.F32_STEP * mag, T)


CASES = [(2, 8, 3, 1024, 144, 2, False, False), (4, 16, 16, 1152, 528, 4, False, True),
         (4, 16, 64, 1152, 528, 4, True, False), (2, 64, 40, 2048, 256, 8, True, True)]


@pytest.mark.parametrize("case", CASES)
def test_stages(case):
    layer = Layer(*case, seed=case[3])
    r = layer.run()
    torch.cuda.synchronize()
    layer.check(r)


@pytest.mark.parametrize("case", CASES[1:3])
def test_side_stream_without_waiting(case):
    layer = Layer(*case, seed=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = layer.run()
        layer.new_inputs()
        second = layer.run(stream=s)
    s.synchronize()
    layer.check(second)
    assert not torch.equal(first["out"], second["out"])


@pytest.mark.parametrize("case", CASES[1:3])
def test_graph_replays_follow_their_inputs(case):
    layer = Layer(*case, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.run()                                        # whatever is made once is made here
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        r = layer.run()
    for _ in range(4):
        layer.new_inputs()
        graph.replay()
        torch.cuda.synchronize()
        layer.check(r)
        eager = layer.run()
        torch.cuda.synchronize()
        for k in ("residual_out", "y", "codes", "dynamic_scales", "shared", "ids", "w", "out"):
            assert torch.equal(r[k], eager[k]), k


def test_two_streams_at_once():
    layers = [Layer(*CASES[1], seed=3), Layer(*CASES[2], seed=4)]
    want = [layer.run()["out"].clone() for layer in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                outs.append(layer.run()["out"])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_plans_and_graphs_that_share_a_workspace():
    """Two plans with one workspace, one after the other on a stream, eager and captured."""
    a, b = Layer(*CASES[0], seed=5), Layer(2, 32, 30, 1024, 144, 2, False, seed=6)
    ex = cq.make_experts(144, BLOCK)
    n = max(cq.moe_dc_experts_layer_workspace_bytes(c.cfg, ex) for c in (a, b))
    ws = torch.empty((n,), dtype=torch.uint8, device=DEV)
    plans, want = [], []
    for c in (a, b):
        r = c.run()
        want.append(cq.experts_layer(c.cfg, ex, r["y"], r["ids"], r["w"], c.up, c.down, up_scales=c.ups,
                                     down_scales=c.downs))
        plans.append(cq.prepare_experts_layer(c.cfg, ex, r["y"], r["ids"], r["w"], c.up, c.down,
                                              up_scales=c.ups, down_scales=c.downs, workspace=ws))
    torch.cuda.synchronize()
    graphs = []
    for launch, _ in plans:
        graphs.append(torch.cuda.CUDAGraph())
        s = torch.cuda.Stream()
        with torch.cuda.graph(graphs[-1], stream=s):
            launch()
    for _ in range(3):
        for i in (0, 1, 1, 0):
            plans[i][1].zero_()
            graphs[i].replay()
            plans[1 - i][0]()
            torch.cuda.synchronize()
            assert torch.equal(plans[i][1], want[i]) and torch.equal(plans[1 - i][1], want[1 - i])


@pytest.mark.parametrize("T", [2, 24])
def test_layer_of_few_tokens_and_separate_calls_agree(T):
    """The same bf16 weights through the layer and through dispatch, two products and combine: both
    round h and y once (the separate calls round o too), so they differ by rounding alone."""
    W, E, H, F, K = 2, 8, 1024, 272, 3
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    cfg = cq.make_config(W, E, T // W, H, K)
    x = torch.randn((W, T // W, H), generator=g, device=DEV).bfloat16()
    logits = torch.randn((W, T // W, E), generator=g, device=DEV)
    up = (torch.randn((E, 2 * F, H), generator=g, device=DEV) / math.sqrt(H)).bfloat16()
    down = (torch.randn((E, H, F), generator=g, device=DEV) / math.sqrt(F)).bfloat16()
    ids, w = cq.gate_topk(cfg, cq.make_gate(renormalize=True), logits)
    y = cq.experts_layer(cfg, cq.make_experts(F), x, ids, w, up, down)
    d = cq.dispatch(cfg, x, ids)
    h = cq.grouped_matmul(cfg, cq.make_matmul(H, 2 * F, activation=SWIGLU), d["expand_x"], up,
                          d["ep_recv_count"], d["recv_offsets"])
    o = cq.grouped_matmul(cfg, cq.make_matmul(F, H), h, down, d["ep_recv_count"], d["recv_offsets"])
    z = cq.combine(cfg, o, ids, d["expand_idx"], w, d["ep_recv_count"], d["recv_offsets"])
    torch.cuda.synchronize()
    # relative to the norm: h, o (one side) and y, half a step each, on both sides
    assert (y.double() - z.double()).norm() <= 5 * 2.0 ** -8 * z.double().norm()
