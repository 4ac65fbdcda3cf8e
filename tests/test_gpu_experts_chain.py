"""The router, dispatch, the experts' products and combine run together, as a layer runs them: on a
side stream without synchronising, from plans, captured in graphs, with empty batches, and several
at once.  Every stage is compared with the plain 64-bit form of its actual inputs."""
import math

import pytest
import torch

import combine_quant_amd as cq
import experts_ref as ref

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Layer:
    """A mixture-of-experts layer on one GPU: router, two products per expert, combine."""

    def __init__(self, W, E, BS, H, I, K, first, second, f16=False, seed=0, mask_kind=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g, self.I, self.first, self.second = g, I, first, second
        token = torch.float16 if f16 else torch.bfloat16
        mode, out_dtype, fmt = {"token": (0, 0, 0), "int8": (2, 0, 0), "e4m3": (2, 2, 0),
                                "mx": (4, 2, 1)}[first]
        self.cfg = cq.make_config(W, E, BS, H, K, mode, out_dtype=out_dtype, scale_format=fmt,
                                  mask_kind=mask_kind,
                                  token_dtype=cq.MOE_TOKEN_F16 if f16 else cq.MOE_TOKEN_BF16)
        self.gate = cq.make_gate(cq.MOE_SCORE_SIGMOID, 4, 2, 2, True, 1.5)
        self.logits = torch.randn((W, BS, E), generator=g, device=DEV)
        self.bias = torch.randn((E,), generator=g, device=DEV) * 0.1
        self.x = torch.randn((W, BS, H), generator=g, device=DEV).to(token)
        self.mask = torch.ones((W, BS), dtype=torch.uint8, device=DEV) if mask_kind else None
        v = torch.randn((E, 2 * I, H), generator=g, device=DEV) / math.sqrt(H)
        self.w1s = None
        if first == "token":
            self.w1 = v.to(token)
            self.mm1 = cq.make_matmul(H, 2 * I, activation=cq.MOE_ACT_SWIGLU)
        elif first == "mx":
            e = torch.frexp(v.view(E, 2 * I, -1, 32).abs().amax(-1)).exponent - 9
            self.w1 = torch.ldexp(v.view(E, 2 * I, -1, 32), -e[..., None]).clamp(-448, 448).view(
                E, 2 * I, H).to(torch.float8_e4m3fn)
            self.w1s = (e + 127).to(torch.uint8)
            self.mm1 = cq.make_matmul(H, 2 * I, x_dtype=cq.MOE_DTYPE_E4M3,
                                      scaling=cq.MOE_MM_SCALE_MX, activation=cq.MOE_ACT_SWIGLU)
        else:
            top = 127.0 if first == "int8" else 448.0
            self.w1s = v.abs().amax(-1) / top
            q = v / self.w1s[..., None]
            self.w1 = q.round().to(torch.int8) if first == "int8" else q.clamp(-448, 448).to(
                torch.float8_e4m3fn)
            self.mm1 = cq.make_matmul(H, 2 * I, x_dtype=cq.MOE_DTYPE_INT8 if first == "int8" else
                                      cq.MOE_DTYPE_E4M3, scaling=cq.MOE_MM_SCALE_ROW,
                                      activation=cq.MOE_ACT_SWIGLU)
        self.w2s = None
        if second == "token":
            self.w2 = (torch.randn((E, H, I), generator=g, device=DEV) / math.sqrt(I)).to(token)
            self.mm2 = cq.make_matmul(I, H)
        else:
            self.w2 = torch.randint(0, 256, (E, H, I // 2), generator=g, device=DEV,
                                    dtype=torch.uint8)
            if second == "int4":
                self.w2s = ((0.5 + torch.rand((E, H, I // 64), generator=g, device=DEV)) /
                            (4.6 * math.sqrt(I))).to(token)
                self.mm2 = cq.make_matmul(I, H, weight_dtype=cq.MOE_W4_INT4, group_size=64)
            else:
                self.w2s = torch.randint(119, 124, (E, H, I // 32), generator=g,
                                         device=DEV).to(torch.uint8)
                self.mm2 = cq.make_matmul(I, H, weight_dtype=cq.MOE_W4_E2M1, group_size=32)

    def run(self, stream=None):
        cfg = self.cfg
        ids, w = cq.gate_topk(cfg, self.gate, self.logits, self.bias, stream=stream)
        d = cq.dispatch(cfg, self.x, ids, x_active_mask=self.mask, stream=stream)
        h = cq.grouped_matmul(cfg, self.mm1, d["expand_x"], self.w1, d["ep_recv_count"],
                              d["recv_offsets"], x_scales=d["dynamic_scales"],
                              weight_scales=self.w1s, stream=stream)
        if self.second == "token":
            o = cq.grouped_matmul(cfg, self.mm2, h, self.w2, d["ep_recv_count"],
                                  d["recv_offsets"], stream=stream)
        else:
            o = cq.grouped_matmul_w4(cfg, self.mm2, h, self.w2, self.w2s, d["ep_recv_count"],
                                     d["recv_offsets"], stream=stream)
        y = cq.combine(cfg, o, ids, d["expand_idx"], w, d["ep_recv_count"], d["recv_offsets"],
                       self.mask, stream=stream)
        return dict(ids=ids, w=w, d=d, h=h, o=o, y=y)

    def ranges(self, d):
        W, E = self.cfg.W, self.cfg.E
        off, erc = d["recv_offsets"].tolist(), d["ep_recv_count"].cpu()
        ends = [off[e // self.cfg.L] + int(erc[e // self.cfg.L, (e % self.cfg.L + 1) * W - 1])
                for e in range(E)]
        return list(zip([0] + ends[:-1], ends)), off[-1]

    def check(self, r):
        cfg, d = self.cfg, r["d"]
        T, K, E = cfg.W * cfg.bs, cfg.topk, cfg.E
        rid, rw = ref.gate(self.logits.view(T, E).cpu(), self.bias.cpu(), K, True, 4, 2, 2, True, 1.5)
        assert torch.equal(r["ids"].view(T, K).cpu(), rid)
        ranges, rows = self.ranges(d)
        assert rows == (T * K if self.mask is None else int(self.mask.sum()) * K)
        # each row went to the expert the router named, from the token it names
        a = d["assist_info"][:rows].long()
        owner = torch.zeros(rows, dtype=torch.long, device=DEV)
        for e, (lo, hi) in enumerate(ranges):
            owner[lo:hi] = e
        assert torch.equal(r["ids"].long()[a[:, 0], a[:, 1], a[:, 2]], owner)
        codes, scales = d["expand_x"][:rows], d["dynamic_scales"]
        if self.first in ("e4m3", "mx"):
            codes = codes.view(torch.float8_e4m3fn)
        xs = None if scales is None else scales[:rows]
        y, err = ref.product(ref.codes_to_f64(codes, xs), ref.codes_to_f64(self.w1, self.w1s),
                             ranges, True, cut=self.first in ("e4m3", "mx"))
        ref.check(r["h"], y, err, rows)
        h = r["h"][:rows].double()
        if self.second == "token":
            y, err = ref.product(h, self.w2.double(), ranges, False)
        else:
            group = 64 if self.second == "int4" else 32
            v = ref.w4_to_f64(self.w2, self.w2s, self.second, group)
            surplus = None
            if self.second == "int4" and r["h"].dtype == torch.bfloat16:
                surplus = (288.0 * self.w2s.double().repeat_interleave(group, 2) * (group + 16) /
                           (self.I + 16) + v.abs())
            y, err = ref.product(h, v, ranges, False, surplus)
        ref.check(r["o"], y, err, rows)
        # combine: the K rows of a token, weighted; K products and sums in fp32, one rounding
        o = r["o"].double()
        back = torch.full((T, K), -1, dtype=torch.long, device=DEV)
        back[a[:, 0] * cfg.bs + a[:, 1], a[:, 2]] = torch.arange(rows, device=DEV)
        w = r["w"].view(T, K).double()
        terms = w[..., None] * o[back.clamp_min(0)] * (back >= 0)[..., None]
        total, mag = terms.sum(1), terms.abs().sum(1)
        err = (K + 2) * ref.F32_STEP * mag
        ref.check(r["y"].view(T, -1), total, err, T)


CASES = [
    dict(W=2, E=16, BS=33, H=1024, I=256, K=4, first="token", second="token"),
    dict(W=2, E=16, BS=33, H=1024, I=320, K=4, first="token", second="int4", f16=True),
    dict(W=4, E=16, BS=40, H=1040, I=256, K=3, first="int8", second="int4"),
    dict(W=2, E=16, BS=64, H=1152, I=256, K=8, first="mx", second="e2m1"),
    dict(W=2, E=8, BS=200, H=1024, I=192, K=2, first="e4m3", second="token"),
    # enough rows and columns for the tile kernels of both products
    dict(W=4, E=32, BS=256, H=2048, I=512, K=4, first="int8", second="int4"),
    dict(W=4, E=32, BS=256, H=2048, I=512, K=4, first="mx", second="e2m1"),
    dict(W=4, E=32, BS=256, H=2048, I=512, K=4, first="token", second="token", f16=True),
    # one token on each rank
    dict(W=2, E=64, BS=1, H=1024, I=256, K=8, first="token", second="int4"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['first']}-{c['second']}-{c['BS']}x{c['E']}")
def test_layer_on_a_side_stream(case):
    layer = Layer(seed=3, **case)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    r = layer.run(stream)
    torch.cuda.current_stream().wait_stream(stream)
    layer.check(r)


def test_layer_against_the_dense_form():
    """The whole layer against 64 bits from its inputs alone; the bound adds up the roundings of
    every stage (2^-8 of h, of o and of y; the fp32 sums)."""
    layer = Layer(W=2, E=8, BS=20, H=1024, I=256, K=2, first="token", second="token", seed=1)
    r = layer.run()
    T, K, I = 40, 2, 256
    x = layer.x.view(T, -1).double()
    w = r["w"].view(T, K).double()
    y = torch.zeros_like(x)
    bound = torch.zeros_like(x)
    half = 2.0 ** -8
    for k in range(K):
        e = r["ids"].view(T, K)[:, k].long()
        w1, w2 = layer.w1.double()[e], layer.w2.double()[e]
        s = torch.matmul(w1, x[:, :, None]).squeeze(2)
        d = (1024 + 16) * ref.F32_STEP * torch.matmul(w1.abs(), x.abs()[:, :, None]).squeeze(2)
        g, u, dg, du = s[:, :I], s[:, I:], d[:, :I], d[:, I:]
        silu = g * torch.sigmoid(g)
        h = silu * u
        dh = 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -17 * h.abs()
        dh = dh + half * (h.abs() + dh)
        o = torch.matmul(w2, h[:, :, None]).squeeze(2)
        do = torch.matmul(w2.abs(), dh[:, :, None]).squeeze(2) + (I + 16) * ref.F32_STEP * torch.matmul(
            w2.abs(), h.abs()[:, :, None]).squeeze(2)
        do = do + half * (o.abs() + do)
        y += w[:, k, None] * o
        bound += w[:, k, None] * do + 4 * ref.F32_STEP * w[:, k, None] * o.abs()
    bound = bound + half * (y.abs() + bound)
    assert ((r["y"].view(T, -1).double() - y).abs() <= bound).all()


@pytest.mark.parametrize("case", [CASES[2], CASES[5], CASES[6], CASES[8]],
                         ids=lambda c: f"{c['first']}-{c['second']}-{c['BS']}x{c['E']}")
def test_layer_in_a_graph(case):
    """A captured layer replayed over inputs changed in place gives the eager layer's bytes; two
    graphs of two layers take turns."""
    layers = [Layer(seed=5, **case), Layer(seed=6, **case)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for layer in layers:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer.run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(layer.run())
        graphs.append(g)
    for turn in range(3):
        for layer, g, out in zip(layers, graphs, outs):
            layer.x.copy_(torch.randn(layer.x.shape, generator=layer.g, device=DEV))
            layer.logits.copy_(torch.randn(layer.logits.shape, generator=layer.g, device=DEV))
            for k in ("h", "o", "y"):
                out[k].fill_(math.nan)
            g.replay()
            eager = layer.run()
            torch.cuda.synchronize()
            rows = int(eager["d"]["recv_offsets"][-1])
            assert torch.equal(out["ids"], eager["ids"]) and torch.equal(out["w"], eager["w"])
            for k in ("h", "o"):
                assert torch.equal(out[k][:rows], eager[k][:rows]), (turn, k)
            assert torch.equal(out["y"], eager["y"]), turn


def test_layers_on_several_streams_at_once():
    layers = [Layer(seed=10 + i, **c) for i, c in enumerate((CASES[2], CASES[3], CASES[5], CASES[7]))]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    results = [layer.run(s) for _ in range(3) for layer, s in zip(layers, streams)][-4:]
    torch.cuda.synchronize()
    for layer, r in zip(layers, results):
        layer.check(r)


@pytest.mark.parametrize("first,second", [("token", "token"), ("int8", "int4"), ("mx", "e2m1")])
def test_masked_tokens_and_an_empty_batch(first, second):
    """Inactive tokens have no rows; without any active token nothing is written."""
    layer = Layer(W=2, E=16, BS=24, H=1024, I=256, K=4, first=first, second=second, seed=8,
                  mask_kind=1)
    layer.mask[:, 5:] = 0
    layer.check(layer.run())
    layer.mask.zero_()
    ids, w = cq.gate_topk(layer.cfg, layer.gate, layer.logits, layer.bias)
    d = cq.dispatch(layer.cfg, layer.x, ids, x_active_mask=layer.mask)
    assert int(d["recv_offsets"][-1]) == 0
    token = cq.token_torch_dtype(layer.cfg)
    out = torch.full((layer.cfg.expand_rows_capacity, 256), 3.5, dtype=token, device=DEV)
    cq.grouped_matmul(layer.cfg, layer.mm1, d["expand_x"], layer.w1, d["ep_recv_count"],
                      d["recv_offsets"], x_scales=d["dynamic_scales"], weight_scales=layer.w1s,
                      out=out)
    o2 = torch.full((layer.cfg.expand_rows_capacity, 1024), 3.5, dtype=token, device=DEV)
    if second != "token":
        cq.grouped_matmul_w4(layer.cfg, layer.mm2, out, layer.w2, layer.w2s, d["ep_recv_count"],
                             d["recv_offsets"], out=o2)
    torch.cuda.synchronize()
    assert (out == 3.5).all() and (o2 == 3.5).all()


def test_plans_launch_again_over_new_contents():
    layer = Layer(seed=9, **CASES[5])
    d = layer.run()["d"]
    run_mm, out = cq.prepare_grouped_matmul(layer.cfg, layer.mm1, d["expand_x"], layer.w1,
                                            d["ep_recv_count"], d["recv_offsets"],
                                            x_scales=d["dynamic_scales"], weight_scales=layer.w1s)
    run_w4, out2 = cq.prepare_grouped_matmul_w4(layer.cfg, layer.mm2, out, layer.w2, layer.w2s,
                                                d["ep_recv_count"], d["recv_offsets"])
    run_gate, (ids, w) = cq.prepare_gate_topk(layer.cfg, layer.gate, layer.logits, layer.bias)
    for turn in range(3):
        layer.logits.copy_(torch.randn(layer.logits.shape, generator=layer.g, device=DEV))
        layer.x.copy_(torch.randn(layer.x.shape, generator=layer.g, device=DEV))
        stream = torch.cuda.Stream() if turn == 1 else None
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        run_gate(stream)
        cq.dispatch(layer.cfg, layer.x, ids, out=d, stream=stream)
        run_mm(stream)
        run_w4(stream)
        y = cq.combine(layer.cfg, out2, ids, d["expand_idx"], w, d["ep_recv_count"],
                       d["recv_offsets"], stream=stream)
        torch.cuda.synchronize()
        layer.check(dict(ids=ids, w=w, d=d, h=out, o=out2, y=y))


def test_the_same_call_gives_the_same_bytes():
    for case in CASES[5:8]:
        layer = Layer(seed=12, **case)
        a, b = layer.run(), layer.run()
        torch.cuda.synchronize()
        rows = int(a["d"]["recv_offsets"][-1])
        assert torch.equal(a["h"][:rows], b["h"][:rows]) and torch.equal(a["o"][:rows], b["o"][:rows])


def test_binding_checks_shapes_and_types():
    layer = Layer(seed=13, **CASES[0])
    d = layer.run()["d"]
    good = dict(x=d["expand_x"], weight=layer.w1, ep_recv_count=d["ep_recv_count"],
                recv_offsets=d["recv_offsets"])

    def call(mm=layer.mm1, **kw):
        cq.grouped_matmul(layer.cfg, mm, **dict(good, **kw))

    with pytest.raises(TypeError):
        call(x=d["expand_x"].float())
    with pytest.raises(ValueError):
        call(x=d["expand_x"][:-1])
    with pytest.raises(ValueError):
        call(weight=layer.w1.transpose(1, 2))
    with pytest.raises(ValueError):
        call(ep_recv_count=d["ep_recv_count"][:1])
    with pytest.raises(TypeError):
        call(recv_offsets=d["recv_offsets"].int())
    with pytest.raises(ValueError):
        call(out=torch.empty((4, 4), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(cq.MoeDcError) as err:
        call(x_scales=torch.ones(layer.cfg.expand_rows_capacity, device=DEV),
             weight_scales=torch.ones((16, 512), device=DEV))
    assert err.value.status == cq.MOE_ERR_INVALID_ARG
    flat = torch.empty(layer.w1.numel() + 8, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(cq.MoeDcError):                    # 2 bytes off a 16-byte boundary
        call(weight=flat[1:1 + layer.w1.numel()].view(layer.w1.shape))
    with pytest.raises(TypeError):
        cq.gate_topk(layer.cfg, layer.gate, layer.logits.bfloat16())
