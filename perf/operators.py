"""Measured cases of the operators around dispatch and combine: the router (gate_topk) and the
experts' products (grouped_matmul, grouped_matmul_w4).

Every case is one call on rows packed as dispatch leaves them: one stable sort of the routed
picks by expert, with ep_recv_count [W][L*W] and recv_offsets [W+1] saying where each expert's
rows begin.  `run` computes the operator either by elementary torch operations in 32 bits
(own = False) or by the library's call (own = True).
"""
import math

import torch

own = False

_DEV = "cuda"
_TOKEN = {"bf16": torch.bfloat16, "f16": torch.float16}
# row types of grouped_matmul: element type of the rows, element type of the weights
_CODES = {"bf16": (torch.bfloat16, torch.bfloat16), "f16": (torch.float16, torch.float16),
          "int8": (torch.int8, torch.int8),
          "e4m3": (torch.float8_e4m3fn, torch.float8_e4m3fn),
          "e5m2": (torch.float8_e5m2, torch.float8_e4m3fn),
          "mx_e4m3": (torch.float8_e4m3fn, torch.float8_e4m3fn),
          "mx_e5m2": (torch.float8_e5m2, torch.float8_e4m3fn)}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# -- cases --------------------------------------------------------------------------------

def _gate(name, W, BS, n, K, score, bias, groups, keep, top, renorm, factor):
    return dict(name=name, op="gate", W=W, BS=BS, n=n, K=K, score=score, bias=bias,
                groups=groups, keep=keep, top=top, renorm=renorm, factor=factor)


def _mm(name, W, E, BS, K, din, dout, type, swiglu, routing="uniform"):
    return dict(name=name, op="mm", W=W, E=E, BS=BS, K=K, din=din, dout=dout, type=type,
                swiglu=swiglu, routing=routing)


def _w4(name, W, E, BS, K, din, dout, type, weight, group, swiglu, routing="uniform"):
    return dict(name=name, op="w4", W=W, E=E, BS=BS, K=K, din=din, dout=dout, type=type,
                weight=weight, group=group, swiglu=swiglu, routing=routing)


def listed():
    return [
        # the router of one decode step: one token on each of two ranks, 256 experts
        _gate("gate_decode", 2, 1, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # the router of the throughput shape: 16 ranks x 512 tokens, 256 experts, top 8
        _gate("gate_w16_bs512", 16, 512, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # plain softmax over 512 routed and 4 special experts, top 16, fp32 logits
        _gate("gate_w32_softmax", 32, 512, 516, 16, "softmax", False, 1, 1, 1, False, 1.0),
        # the tiny round trip's expert product: 64 rows on 8 experts (latency)
        _mm("mm_bf16_tiny", 2, 8, 16, 2, 1024, 1024, "bf16", True),
        # decode of the sample table's low-latency shape: 64 tokens, 32 experts, gate and up
        _mm("mm_bf16_decode", 8, 32, 8, 8, 7168, 4096, "bf16", True),
        # the sample table's throughput shape, gate and up in bf16: about 512 rows an expert
        _mm("mm_bf16_w8_bs256", 8, 32, 256, 8, 7168, 4096, "bf16", True),
        # odd sizes in fp16: 37 tokens on 3 ranks, 777 outputs, inner size a multiple of 8 only
        _mm("mm_f16_odd", 3, 12, 37, 3, 1144, 777, "f16", False),
        # the down product on E4M3 codes with row scales, 8 ranks x 128 tokens on 256 experts
        _mm("mm_e4m3_w8_bs128", 8, 256, 128, 8, 2048, 7168, "e4m3", False),
        # int8 rows of the round-trip workload (16 ranks x 512 tokens, 256 experts), gate and up
        _mm("mm_int8_w16_bs512", 16, 256, 512, 8, 7168, 4096, "int8", True),
        # MX E4M3 rows of the skewed workload: few experts hold most rows
        _mm("mm_mx_w16_zipf", 16, 256, 512, 8, 7168, 4096, "mx_e4m3", True, "zipf"),
        # one token on each of two ranks: 16 matrix-vector products with int4 weights
        _w4("w4_int4_single", 2, 64, 1, 8, 7168, 4096, "bf16", "int4", 128, True),
        # the down product of a prompt chunk with MX E2M1 weights: about 128 rows an expert
        _w4("w4_e2m1_w8_bs64", 8, 32, 64, 8, 2048, 7168, "bf16", "e2m1", 32, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MAX_FLOPS = 3.5e12        # below the largest listed products
_MAX_WEIGHTS = 4.0e9       # elements of all experts' weights


def draw(rng):
    op = rng.choice(("gate", "mm", "mm", "w4"))
    W = rng.choice((2, 3, 4, 5, 8, 12, 16))
    if op == "gate":
        groups = rng.choice((1, 1, 2, 4, 8))
        n = groups * _log(rng, max(2, 16 // groups), 1024 // groups)
        keep = rng.randint(1, groups)
        top = rng.choice((1, 2)) if groups > 1 else 1
        K = rng.randint(1, min(16, n // groups * keep))
        score = rng.choice(("softmax", "sigmoid"))
        return dict(op="gate", W=W, BS=_log(rng, 1, 512), n=n, K=K, score=score,
                    bias=rng.random() < 0.5, groups=groups, keep=keep, top=top,
                    renorm=rng.random() < 0.5, factor=rng.choice((1.0, 2.5)))
    E = W * max(1, _log(rng, 1, 256) // W)
    K = rng.randint(1, min(8, E))
    BS = _log(rng, 1, 512)
    dout = _log(rng, 48, 8192)
    swiglu = rng.random() < 0.5
    if swiglu:
        dout += dout % 2
    routing = rng.choice(("uniform", "uniform", "zipf"))
    if op == "mm":
        kind = rng.choice(("bf16", "bf16", "f16", "int8", "e4m3", "e5m2", "mx_e4m3", "mx_e5m2"))
        step = 128 if kind.startswith("mx") else 8 if kind in _TOKEN else 16
        case = dict(op="mm", type=kind)
    else:
        weight = rng.choice(("int4", "e2m1"))
        group = 32 if weight == "e2m1" else rng.choice((32, 64, 128))
        step = group
        case = dict(op="w4", type=rng.choice(("bf16", "f16")), weight=weight, group=group)
    din = step * max(1, _log(rng, 128, 8192) // step)
    while E * dout * din > _MAX_WEIGHTS and E > W:
        E -= W * ((E // W + 1) // 2)
    K = min(K, E)
    while 2.0 * W * BS * K * din * dout > _MAX_FLOPS and BS > 1:
        BS = BS // 2
    case.update(W=W, E=E, BS=BS, K=K, din=din, dout=dout, swiglu=swiglu, routing=routing)
    return case


# -- inputs -------------------------------------------------------------------------------

def _generator(seed, part):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed * 16 + part)
    return g


def _routing(case, seed):
    """Rows per (expert, source rank) of K distinct experts a token, uniform or Zipf(1.2) over
    a seeded order of the experts; returned as dispatch returns them, and on the host."""
    W, E, BS, K = case["W"], case["E"], case["BS"], case["K"]
    T = W * BS
    g = _generator(seed, 0)
    keys = -torch.log(-torch.log(torch.rand((T, E), generator=g, device=_DEV).clamp(1e-20, 1 - 1e-7)))
    if case["routing"] == "zipf":
        rank = torch.randperm(E, generator=g, device=_DEV) + 1
        keys = keys - 1.2 * torch.log(rank.float())
    ids = torch.topk(keys, K, dim=1).indices
    source = torch.arange(T, device=_DEV).div(BS, rounding_mode="floor")[:, None]
    counts = torch.bincount((ids * W + source).flatten(), minlength=E * W)
    per_rank = counts.view(W, (E // W) * W)
    ep_recv_count = per_rank.cumsum(1).to(torch.int32).contiguous()
    recv_offsets = torch.zeros(W + 1, dtype=torch.int64, device=_DEV)
    recv_offsets[1:] = per_rank.sum(1).cumsum(0)
    ends = counts.view(E, W).sum(1).cumsum(0).tolist()
    return ep_recv_count, recv_offsets, list(zip([0] + ends[:-1], ends))


def _mx_quantise(v, codes):
    """fp32 [r][k] -> codes and E8M0 bytes, one per 32: exponent floor(log2 max|v|) - emax."""
    emax, top = (8, 448.0) if codes == torch.float8_e4m3fn else (15, 57344.0)
    b = v.view(v.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True).clamp_min(1e-30)
    e = (torch.frexp(amax).exponent - 1 - emax).clamp_min(-127)
    q = torch.ldexp(b, -e).clamp(-top, top).to(codes)
    return q.view(v.shape), (e.squeeze(2) + 127).to(torch.uint8)


def _row_quantise(v, codes):
    """fp32 [r][k] -> codes and one fp32 scale a row (largest magnitude over the type's)."""
    top = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}[codes]
    s = v.abs().amax(1, keepdim=True) / top
    q = v / s
    q = q.round().clamp(-top, top) if codes == torch.int8 else q.clamp(-top, top)
    return q.to(codes), s.squeeze(1)


def _encode(v, kind, codes):
    if kind in _TOKEN:
        return v.to(codes), None
    return _mx_quantise(v, codes) if kind.startswith("mx") else _row_quantise(v, codes)


def _prepare_gate(case, seed):
    g = _generator(seed, 1)
    T, n = case["W"] * case["BS"], case["n"]
    logits = torch.randn((case["W"], case["BS"], n), generator=g, device=_DEV) * 1.5
    bias = None
    if case["bias"]:
        bias = torch.randn((n,), generator=g, device=_DEV) * 0.05
    st = dict(case=case, logits=logits, bias=bias)
    if own:
        import combine_quant_amd as cq
        special = n % case["W"]                  # routed experts are a multiple of the ranks
        cfg = cq.make_config(case["W"], n - special, case["BS"], 1024, case["K"],
                             zero_expert_num=special)
        gate = cq.make_gate(score=getattr(cq, "MOE_SCORE_" + case["score"].upper()),
                            group_count=case["groups"], group_keep=case["keep"],
                            group_top=case["top"], renormalize=case["renorm"],
                            factor=case["factor"])
        st["launch"], st["out"] = cq.prepare_gate_topk(cfg, gate, logits, bias)
    return st


def _prepare_rows(case, seed):
    """The packed rows: N(0,1) tokens of differing magnitude, encoded as dispatch does."""
    st = dict(case=case)
    st["counts"], st["offsets"], st["ranges"] = _routing(case, seed)
    g = _generator(seed, 2)
    rows, din = case["W"] * case["BS"] * case["K"], case["din"]
    kind = case["type"]
    codes = _CODES[kind][0]
    x = torch.empty((rows, din), dtype=codes, device=_DEV)
    xs = None
    if kind.startswith("mx"):
        xs = torch.empty((rows, din // 32), dtype=torch.uint8, device=_DEV)
    elif kind not in _TOKEN:
        xs = torch.empty((rows,), dtype=torch.float32, device=_DEV)
    for lo in range(0, rows, 8192):
        hi = min(rows, lo + 8192)
        v = torch.randn((hi - lo, din), generator=g, device=_DEV)
        v *= 0.5 + torch.rand((hi - lo, 1), generator=g, device=_DEV)
        q, s = _encode(v, kind, codes)
        x[lo:hi] = q
        if xs is not None:
            xs[lo:hi] = s
    st["x"], st["xs"] = x, xs
    return st


def _prepare_mm(case, seed):
    st = _prepare_rows(case, seed)
    g = _generator(seed, 3)
    E, dout, din, kind = case["E"], case["dout"], case["din"], case["type"]
    codes = _CODES[kind][1]
    w = torch.empty((E, dout, din), dtype=codes, device=_DEV)
    ws = None
    if kind.startswith("mx"):
        ws = torch.empty((E, dout, din // 32), dtype=torch.uint8, device=_DEV)
    elif kind not in _TOKEN:
        ws = torch.empty((E, dout), dtype=torch.float32, device=_DEV)
    for e in range(E):
        v = torch.randn((dout, din), generator=g, device=_DEV) / math.sqrt(din)
        w[e], s = _encode(v, kind, codes)
        if ws is not None:
            ws[e] = s
    st["w"], st["ws"] = w, ws
    if own:
        import combine_quant_amd as cq
        cfg = cq.make_config(case["W"], E, case["BS"], min(max(din, 1024), 8192), case["K"],
                             token_dtype=cq.MOE_TOKEN_F16 if kind == "f16" else cq.MOE_TOKEN_BF16)
        x_dtype = {"bf16": cq.MOE_DTYPE_DEFAULT, "f16": cq.MOE_DTYPE_DEFAULT,
                   "int8": cq.MOE_DTYPE_INT8, "e4m3": cq.MOE_DTYPE_E4M3,
                   "e5m2": cq.MOE_DTYPE_E5M2, "mx_e4m3": cq.MOE_DTYPE_E4M3,
                   "mx_e5m2": cq.MOE_DTYPE_E5M2}[kind]
        mm = cq.make_matmul(din, dout, x_dtype=x_dtype,
                            scaling=cq.MOE_MM_SCALE_MX if kind.startswith("mx")
                            else cq.MOE_MM_SCALE_NONE if kind in _TOKEN else cq.MOE_MM_SCALE_ROW,
                            activation=cq.MOE_ACT_SWIGLU if case["swiglu"] else cq.MOE_ACT_NONE)
        st["launch"], st["out"] = cq.prepare_grouped_matmul(
            cfg, mm, st["x"], w, st["counts"], st["offsets"], x_scales=st["xs"],
            weight_scales=ws)
    return st


def _prepare_w4(case, seed):
    st = _prepare_rows(case, seed)
    g = _generator(seed, 3)
    E, dout, din, group = case["E"], case["dout"], case["din"], case["group"]
    token = _TOKEN[case["type"]]
    w = torch.randint(0, 256, (E, dout, din // 2), generator=g, device=_DEV, dtype=torch.uint8)
    u = torch.rand((E, dout, din // group), generator=g, device=_DEV)
    if case["weight"] == "int4":
        ws = ((0.5 + u) / (4.6 * math.sqrt(din))).to(token)
    else:                            # E8M0: powers of two around 1 / sqrt(din)
        ws = (127 - round(math.log2(3.0 * math.sqrt(din))) + (u * 3).floor() - 1).to(torch.uint8)
    st["w"], st["ws"] = w, ws
    if own:
        import combine_quant_amd as cq
        cfg = cq.make_config(case["W"], E, case["BS"], min(max(din, 1024), 8192), case["K"],
                             token_dtype=cq.MOE_TOKEN_F16 if case["type"] == "f16"
                             else cq.MOE_TOKEN_BF16)
        mm = cq.make_matmul(din, dout,
                            weight_dtype=cq.MOE_W4_INT4 if case["weight"] == "int4"
                            else cq.MOE_W4_E2M1, group_size=group,
                            activation=cq.MOE_ACT_SWIGLU if case["swiglu"] else cq.MOE_ACT_NONE)
        st["launch"], st["out"] = cq.prepare_grouped_matmul_w4(
            cfg, mm, st["x"], w, ws, st["counts"], st["offsets"])
    return st


def prepare(case, seed):
    return {"gate": _prepare_gate, "mm": _prepare_mm, "w4": _prepare_w4}[case["op"]](case, seed)


# -- the operators in plain form ----------------------------------------------------------

def _plain_gate(st):
    """The choice is made in 64 bits: scores next to each other decide which id comes first."""
    case, T, n = st["case"], st["case"]["W"] * st["case"]["BS"], st["case"]["n"]
    z = st["logits"].view(T, n).double()
    score = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, 1)
    choice = score if st["bias"] is None else score + st["bias"].double()
    order = z if st["bias"] is None else choice        # scores rise with the logits
    G = case["groups"]
    if G > 1:
        part = (choice if case["top"] == 2 else order).view(T, G, n // G)
        best = torch.sort(part, dim=2, descending=True).values[:, :, :case["top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        off = torch.ones((T, G), dtype=torch.bool, device=z.device).scatter_(1, kept, False)
        order = order.masked_fill(off.repeat_interleave(n // G, 1), -math.inf)
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :case["K"]]
    weight = torch.gather(score, 1, ids)
    if case["renorm"]:
        weight = weight / (weight.sum(1, keepdim=True) + 1e-20)
    weight = weight * case["factor"]
    shape = (case["W"], case["BS"], case["K"])
    return ids.to(torch.int32).view(shape), weight.float().view(shape)


def _values(codes, scales):
    """Codes and their scales (one a row, or E8M0 bytes per 32) as fp32 values [r][k]."""
    v = codes.float()
    if scales is None:
        return v
    if scales.dtype == torch.uint8:
        s = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
        return (v.view(v.shape[0], -1, 32) * s[:, :, None]).view(v.shape)
    return v * scales[:, None]


def _values_w4(w, ws, kind, group):
    """Two codes a byte (even index low) times their group's scale, as fp32 [n][k]."""
    u = torch.stack((w & 15, w >> 4), 2).view(w.shape[0], -1).int()
    if kind == "int4":
        v, s = (u - 16 * (u >> 3)).float(), ws.float()
    else:
        v = torch.tensor(_E2M1, device=w.device)[u.long()]
        s = torch.ldexp(torch.ones_like(ws, dtype=torch.float32), ws.int() - 127)
    return (v.view(v.shape[0], -1, group) * s[:, :, None]).view(v.shape)


def _plain_product(st):
    case = st["case"]
    rows, dout = st["x"].shape[0], case["dout"]
    token = torch.float16 if case["type"] == "f16" else torch.bfloat16
    out = torch.empty((rows, dout // 2 if case["swiglu"] else dout), dtype=token,
                      device=st["x"].device)
    for e, (lo, hi) in enumerate(st["ranges"]):
        if lo == hi:
            continue
        x = _values(st["x"][lo:hi], None if st["xs"] is None else st["xs"][lo:hi])
        if case["op"] == "w4":
            w = _values_w4(st["w"][e], st["ws"][e], case["weight"], case["group"])
        else:
            w = _values(st["w"][e], None if st["ws"] is None else st["ws"][e])
        y = x @ w.t()
        if case["swiglu"]:
            gate, up = y[:, :dout // 2], y[:, dout // 2:]
            y = gate / (1.0 + torch.exp(-gate)) * up
        out[lo:hi] = y.to(token)
    return out


def run(state):
    if own:
        state["launch"]()
        return state["out"]
    return _plain_gate(state) if state["case"]["op"] == "gate" else _plain_product(state)


# -- what a pass cannot do without ----------------------------------------------------------

def _expected_active(case):
    """Experts expected to have rows: their weights have to be read."""
    T, E, K = case["W"] * case["BS"], case["E"], case["K"]
    if case["routing"] == "zipf":
        p = [r ** -1.2 for r in range(1, E + 1)]
        share = [min(1.0, K * v / sum(p)) for v in p]
    else:
        share = [K / E] * E
    return sum(1.0 - (1.0 - s) ** T for s in share)


def work(case):
    T = case["W"] * case["BS"]
    if case["op"] == "gate":
        return {"bytes": T * case["n"] * 4 + (case["n"] * 4 if case["bias"] else 0)
                + T * case["K"] * 8, "flops": 4 * T * case["n"]}
    rows, din, dout = T * case["K"], case["din"], case["dout"]
    size = {"bf16": 2.0, "f16": 2.0}.get(case["type"], 1.0)
    row = din * size
    if case["type"].startswith("mx"):
        row += din / 32
    elif size == 1.0:
        row += 4
    if case["op"] == "w4":
        weight = din / 2 + din / case["group"] * (2 if case["weight"] == "int4" else 1)
    else:
        weight = row
    out = rows * (dout // 2 if case["swiglu"] else dout) * 2
    return {"bytes": int(rows * row + _expected_active(case) * dout * weight + out),
            "flops": 2 * rows * din * dout}


# -- the definition in 64 bits ----------------------------------------------------------------

def _exact_gate(case, st):
    z = st["logits"].double().reshape(-1, case["n"])
    T, n, G = z.shape[0], case["n"], case["groups"]
    if case["score"] == "softmax":
        e = torch.exp(z - z.max(1, keepdim=True).values)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-z))
    key = z.clone()
    if st["bias"] is not None:
        key = score + st["bias"].double()
    if G > 1:
        value = key if case["top"] == 1 or st["bias"] is not None else score
        members = value.view(T, G, n // G)
        total = torch.zeros((T, G), dtype=torch.float64, device=z.device)
        for _ in range(case["top"]):
            best = members.max(2, keepdim=True)
            total = total + best.values.squeeze(2)
            members = members.scatter(2, best.indices, -math.inf)
        # the groups that at most keep - 1 others precede (larger, or equal and earlier)
        i = torch.arange(G, device=z.device)
        ahead = (total[:, None, :] > total[:, :, None]) | (
            (total[:, None, :] == total[:, :, None]) & (i[None, None, :] < i[None, :, None]))
        stays = ahead.sum(2) < case["keep"]
        key = torch.where(stays[:, :, None].expand(T, G, n // G).reshape(T, n), key, -math.inf)
    ids = []
    for _ in range(case["K"]):
        top = key.max(1, keepdim=True).values
        first = (key == top).to(torch.int8).argmax(1, keepdim=True)
        ids.append(first)
        key = key.scatter(1, first, -math.inf)
    ids = torch.cat(ids, 1)
    weight = score.gather(1, ids)
    if case["renorm"]:
        weight = weight / (weight.sum(1, keepdim=True) + 1e-20)
    shape = (case["W"], case["BS"], case["K"])
    return ids.to(torch.int32).view(shape), (weight * case["factor"]).view(shape)


def _exact_power(b):
    return torch.pow(2.0, b.double() - 127.0)


def _exact_product(case, st):
    dout = case["dout"]
    half = dout // 2
    y = torch.zeros((st["x"].shape[0], half if case["swiglu"] else dout), dtype=torch.float64,
                    device=st["x"].device)
    table = torch.tensor(_E2M1, dtype=torch.float64, device=st["x"].device)
    for e in range(case["E"]):
        lo, hi = st["ranges"][e]
        if hi == lo:
            continue
        a, w = st["x"][lo:hi].double(), st["w"][e]
        if case["op"] == "w4":
            even, odd = torch.remainder(w.int(), 16), torch.div(w.int(), 16, rounding_mode="floor")
            c = torch.empty((dout, case["din"]), dtype=torch.float64, device=w.device)
            if case["weight"] == "int4":
                c[:, 0::2] = torch.where(even > 7, even - 16, even).double()
                c[:, 1::2] = torch.where(odd > 7, odd - 16, odd).double()
                s = st["ws"][e].double()
            else:
                c[:, 0::2], c[:, 1::2] = table[even.long()], table[odd.long()]
                s = _exact_power(st["ws"][e])
            b = c * s.repeat_interleave(case["group"], 1)
        else:
            b = w.double()
            if st["ws"] is not None and st["ws"].dtype == torch.uint8:
                b = b * _exact_power(st["ws"][e]).repeat_interleave(32, 1)
                a = a * _exact_power(st["xs"][lo:hi]).repeat_interleave(32, 1)
        r = torch.mm(a, b.t())
        if st["ws"] is not None and st["ws"].dtype == torch.float32:
            r = r * st["xs"][lo:hi].double()[:, None] * st["ws"][e].double()[None, :]
        if case["swiglu"]:
            r = r[:, :half] * torch.sigmoid(r[:, :half]) * r[:, half:]
        y[lo:hi] = r
    return y


def exact(case, seed):
    global own
    mine, own = own, False           # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    return _exact_gate(case, st) if case["op"] == "gate" else _exact_product(case, st)
