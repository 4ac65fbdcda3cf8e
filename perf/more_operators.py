"""Measured cases of the operators around dispatch's 8-bit rows: the experts' product on rows with a
scale per 128 elements (grouped_matmul with MOE_MM_SCALE_BLOCK), the same product with its results
coded again (grouped_matmul_quantize), the RMS norm that makes the layer's tokens and their codes
(rms_norm), and the experts' layer of a few tokens (experts_layer).

`run` computes an operator either by elementary torch operations in 32 bits (own = False) or by the
library's call (own = True).
"""
import math

import torch

own = False

_DEV = "cuda"
_TOKEN = {"bf16": torch.bfloat16, "f16": torch.float16}
_CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_TOP = {"e4m3": 448.0, "e5m2": 57344.0}
_BLOCK = 128


# -- cases --------------------------------------------------------------------------------

def _block(name, W, E, BS, K, din, dout, rows, swiglu, codes=""):
    """A product of rows in `rows`; `codes`: the type its results are coded in, or none."""
    return dict(name=name, op="codes" if codes else "block", W=W, E=E, BS=BS, K=K, din=din,
                dout=dout, rows=rows, swiglu=swiglu, codes=codes)


def _norm(name, W, BS, H, mode, codes, token, residual):
    """mode 0: tokens alone; 2: one scale a token; 3: one per 128 elements."""
    return dict(name=name, op="norm", W=W, BS=BS, H=H, mode=mode, codes=codes, token=token,
                residual=residual)


def _few(name, W, E, BS, K, H, F, token, weights, active):
    """weights: "token" or "block"; active: tokens that are not masked out."""
    return dict(name=name, op="few", W=W, E=E, BS=BS, K=K, H=H, F=F, token=token,
                weights=weights, active=active)


def listed():
    return [
        # the tiny round trip's product: 64 rows on 8 experts (latency)
        _block("block_tiny", 2, 8, 16, 2, 1024, 1024, "e4m3", True),
        # the sample table's throughput shape, gate and up: about 512 rows an expert
        _block("block_w8_bs256", 8, 32, 256, 8, 7168, 4096, "e4m3", True),
        # the down product of 8 ranks x 128 tokens on 256 experts: bound by the weights' bytes
        _block("block_e5m2_w8_bs128", 8, 256, 128, 8, 2048, 7168, "e5m2", False),
        # odd sizes: 37 tokens on 3 ranks, a last group of 112 elements, 777 outputs
        _block("block_odd", 3, 12, 37, 3, 1136, 777, "e4m3", False),
        # the throughput shape with its results coded for the down product
        _block("codes_w8_bs256", 8, 32, 256, 8, 7168, 4096, "e4m3", True, "e4m3"),
        # odd sizes: 712 columns, coded as E5M2
        _block("codes_odd", 3, 12, 37, 3, 1136, 1424, "e4m3", True, "e5m2"),
        # one decode step's norm: a token on each of two ranks
        _norm("norm_decode", 2, 1, 7168, 2, "e4m3", "bf16", True),
        # a prompt chunk of 16 ranks x 512 tokens, coded for the block-scaled product
        _norm("norm_w16_bs512", 16, 512, 7168, 3, "e4m3", "bf16", True),
        # odd sizes in fp16: 185 tokens, a last group of 8 elements, no residual
        _norm("norm_f16_odd", 5, 37, 5128, 3, "e5m2", "f16", False),
        # decode of a single token (the other rank idles): 8 of 64 experts, bf16 weights
        _few("few_single", 2, 64, 1, 8, 7168, 2048, "bf16", "token", 1),
        # decode of 32 tokens on 256 experts with E4M3 weights: about 160 experts have tokens
        _few("few_block_w8_bs4", 8, 256, 4, 8, 7168, 2048, "bf16", "block", 32),
        # a small fp16 layer on 5 tokens of 8 slots (latency)
        _few("few_f16_tiny", 2, 8, 4, 2, 1024, 520, "f16", "token", 5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_MAX_FLOPS = 0.9e12        # below the largest listed products
_MAX_WEIGHTS = 3.0e9       # elements of all experts' weights
_MAX_FEW = 9.0e9           # elements of the weights of every pick of a layer of a few tokens


def draw(rng):
    op = rng.choice(("block", "block", "codes", "norm", "few", "few"))
    W = rng.choice((2, 3, 4, 5, 8, 12, 16))
    if op == "norm":
        return dict(op="norm", W=W, BS=_log(rng, 1, 512), H=8 * _log(rng, 128, 1024),
                    mode=rng.choice((0, 2, 3, 3)), codes=rng.choice(("e4m3", "e4m3", "e5m2")),
                    token=rng.choice(("bf16", "bf16", "f16")), residual=rng.random() < 0.7)
    E = W * max(1, _log(rng, W, 256) // W)
    K = rng.randint(1, min(8, E))
    if op == "few":
        BS = _log(rng, 1, max(1, 64 // W))
        weights = rng.choice(("token", "block"))
        step = 8 if weights == "token" else 16
        H, F = step * (_log(rng, 1024, 8192) // step), step * (_log(rng, 256, 4096) // step)
        picks = W * BS * K
        while 3 * picks * H * F > _MAX_FEW and F > 256:
            F = step * (F // 2 // step)
        while 3 * E * H * F > _MAX_FEW and E > W:
            E -= W * ((E // W + 1) // 2)
        return dict(op="few", W=W, E=E, BS=BS, K=min(K, E), H=H, F=F,
                    token=rng.choice(("bf16", "bf16", "f16")), weights=weights,
                    active=W * BS if rng.random() < 0.7 else rng.randint(1, W * BS))
    BS = _log(rng, 1, 512)
    din, dout = 16 * _log(rng, 16, 512), _log(rng, 48, 8192)
    swiglu = rng.random() < 0.5
    if swiglu:
        dout += dout % 2
    while E * dout * din > _MAX_WEIGHTS and E > W:
        E -= W * ((E // W + 1) // 2)
    K = min(K, E)
    while 2.0 * W * BS * K * din * dout > _MAX_FLOPS and BS > 1:
        BS = BS // 2
    return dict(op=op, W=W, E=E, BS=BS, K=K, din=din, dout=dout,
                rows=rng.choice(("e4m3", "e4m3", "e5m2")), swiglu=swiglu,
                codes=rng.choice(("e4m3", "e5m2")) if op == "codes" else "")


# -- inputs -------------------------------------------------------------------------------

def _generator(seed, part):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed * 16 + part)
    return g


def _choices(T, E, K, g):
    """K distinct experts a token, all alike."""
    return torch.topk(torch.rand((T, E), generator=g, device=_DEV), K, dim=1).indices


def _routing(case, seed):
    """Rows per (expert, source rank), as dispatch returns them, and each expert's first row and
    number of rows; the most rows an expert has, on the host."""
    W, E, BS, K = case["W"], case["E"], case["BS"], case["K"]
    T = W * BS
    ids = _choices(T, E, K, _generator(seed, 0))
    source = torch.arange(T, device=_DEV).div(BS, rounding_mode="floor")[:, None]
    counts = torch.bincount((ids * W + source).flatten(), minlength=E * W)
    per_rank = counts.view(W, (E // W) * W)
    ep_recv_count = per_rank.cumsum(1).to(torch.int32).contiguous()
    recv_offsets = torch.zeros(W + 1, dtype=torch.int64, device=_DEV)
    recv_offsets[1:] = per_rank.sum(1).cumsum(0)
    per_expert = counts.view(E, W).sum(1)
    return ep_recv_count, recv_offsets, per_expert.cumsum(0) - per_expert, per_expert


def _groups(n):
    return (n + _BLOCK - 1) // _BLOCK


def _code_rows(v, kind):
    """fp32 [r][k] -> codes and one fp32 scale per 128 elements, as dispatch codes a token."""
    r, k = v.shape
    amax = torch.nn.functional.pad(v.abs(), (0, -k % _BLOCK)).view(r, -1, _BLOCK).amax(2)
    dyn = _TOP[kind] / amax
    return (v * _spread(dyn, 1, k)).clamp(-_TOP[kind], _TOP[kind]).to(_CODE[kind]), 1.0 / dyn


def _spread(s, dim, n):
    """One value per 128 places along a dimension -> one per place, n of them."""
    return s.repeat_interleave(_BLOCK, dim).narrow(dim, 0, n)


def _code_weights(v):
    """fp32 [n][k] -> E4M3 codes and one fp32 scale per 128 x 128 block."""
    n, k = v.shape
    p = torch.nn.functional.pad(v.abs(), (0, -k % _BLOCK, 0, -n % _BLOCK))
    s = p.view(_groups(n), _BLOCK, _groups(k), _BLOCK).amax((1, 3)) / 448.0
    return (v / _spread(_spread(s, 0, n), 1, k)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s


def _weights(E, parts, n, k, token, block, g):
    """Weights [E][parts * n][k] of `parts` matrices one above the other, N(0, 1 / k), in the
    token type or as codes with scales [E][parts * ceil(n / 128)][ceil(k / 128)]."""
    w = torch.empty((E, parts, n, k), dtype=torch.float8_e4m3fn if block else token, device=_DEV)
    s = torch.empty((E, parts, _groups(n), _groups(k)), device=_DEV) if block else None
    for e in range(E):
        for p in range(parts):
            v = torch.randn((n, k), generator=g, device=_DEV) / math.sqrt(k)
            if block:
                w[e, p], s[e, p] = _code_weights(v)
            else:
                w[e, p] = v.to(token)
    return w.view(E, parts * n, k), s.view(E, -1, _groups(k)) if block else None


def _prepare_block(case, seed):
    st = dict(case=case)
    st["counts"], st["offsets"], st["first"], st["many"] = _routing(case, seed)
    st["most"] = int(st["many"].max())
    rows, din, kind = case["W"] * case["BS"] * case["K"], case["din"], case["rows"]
    g = _generator(seed, 1)
    x = torch.empty((rows, din), dtype=_CODE[kind], device=_DEV)
    xs = torch.empty((rows, _groups(din)), device=_DEV)
    for lo in range(0, rows, 8192):
        hi = min(rows, lo + 8192)
        v = torch.randn((hi - lo, din), generator=g, device=_DEV)
        v *= 0.5 + torch.rand((hi - lo, 1), generator=g, device=_DEV)
        x[lo:hi], xs[lo:hi] = _code_rows(v, kind)
    st["x"], st["xs"] = x, xs
    parts = 2 if case["swiglu"] else 1
    st["w"], st["ws"] = _weights(case["E"], parts, case["dout"] // parts, din, None, True,
                                 _generator(seed, 2))
    if own:
        import combine_quant_amd as cq
        cfg = cq.make_config(case["W"], case["E"], case["BS"], min(max(din, 1024), 8192), case["K"])
        types = {"e4m3": cq.MOE_DTYPE_E4M3, "e5m2": cq.MOE_DTYPE_E5M2}
        mm = cq.make_matmul(din, case["dout"], x_dtype=types[kind], scaling=cq.MOE_MM_SCALE_BLOCK,
                            activation=cq.MOE_ACT_SWIGLU if case["swiglu"] else cq.MOE_ACT_NONE)
        if case["codes"]:
            st["launch"], st["out"] = cq.prepare_grouped_matmul_quantize(
                cfg, mm, types[case["codes"]], x, xs, st["w"], st["ws"], st["counts"], st["offsets"])
        else:
            st["launch"], st["out"] = cq.prepare_grouped_matmul(
                cfg, mm, x, st["w"], st["counts"], st["offsets"], x_scales=xs, weight_scales=st["ws"])
    return st


def _prepare_norm(case, seed):
    g = _generator(seed, 3)
    shape, token = (case["W"], case["BS"], case["H"]), _TOKEN[case["token"]]
    st = dict(case=case)
    st["x"] = (torch.randn(shape, generator=g, device=_DEV)).to(token)
    # the residual stream has grown over the layers, by a factor that differs from token to token
    st["residual"] = (torch.randn(shape, generator=g, device=_DEV) * (1.0 + 7.0 * torch.rand(
        shape[:2] + (1,), generator=g, device=_DEV))).to(token) if case["residual"] else None
    st["gamma"] = (0.5 + torch.rand(shape[2:], generator=g, device=_DEV)).to(token)
    if own:
        import combine_quant_amd as cq
        cfg = cq.make_config(case["W"], case["W"], case["BS"], case["H"], 1, quant_mode=case["mode"],
                             out_dtype=cq.MOE_DTYPE_DEFAULT if case["mode"] == 0 else
                             {"e4m3": cq.MOE_DTYPE_E4M3, "e5m2": cq.MOE_DTYPE_E5M2}[case["codes"]],
                             token_dtype=cq.MOE_TOKEN_F16 if case["token"] == "f16"
                             else cq.MOE_TOKEN_BF16)
        st["launch"], st["out"] = cq.prepare_rms_norm(cfg, cq.make_norm(1e-6), st["x"], st["gamma"],
                                                      residual=st["residual"])
    return st


def _prepare_few(case, seed):
    g = _generator(seed, 4)
    W, E, BS, K, H, F = (case[k] for k in ("W", "E", "BS", "K", "H", "F"))
    T, token, block = W * BS, _TOKEN[case["token"]], case["weights"] == "block"
    st = dict(case=case)
    st["x"] = torch.randn((W, BS, H), generator=g, device=_DEV).to(token)
    st["ids"] = _choices(T, E, K, g).to(torch.int32).view(W, BS, K)
    weight = torch.rand((W, BS, K), generator=g, device=_DEV)
    st["weight"] = weight / weight.sum(2, keepdim=True)
    st["mask"] = None
    if case["active"] < T:
        st["mask"] = (torch.randperm(T, generator=g, device=_DEV) < case["active"]).view(W, BS)
    st["up"], st["ups"] = _weights(E, 2, F, H, token, block, g)
    st["down"], st["downs"] = _weights(E, 1, H, F, token, block, g)
    if own:
        import combine_quant_amd as cq
        cfg = cq.make_config(W, E, BS, H, K, mask_kind=0 if st["mask"] is None else 1,
                             token_dtype=cq.MOE_TOKEN_F16 if case["token"] == "f16"
                             else cq.MOE_TOKEN_BF16)
        experts = cq.make_experts(F, scaling=cq.MOE_MM_SCALE_BLOCK if block else cq.MOE_MM_SCALE_NONE)
        st["launch"], st["out"] = cq.prepare_experts_layer(
            cfg, experts, st["x"], st["ids"], st["weight"], st["up"], st["down"],
            up_scales=st["ups"], down_scales=st["downs"], x_active_mask=st["mask"])
    return st


def prepare(case, seed):
    return {"block": _prepare_block, "codes": _prepare_block, "norm": _prepare_norm,
            "few": _prepare_few}[case["op"]](case, seed)


# -- the operators in plain form ----------------------------------------------------------

def _values(w, s, parts):
    """Weights [..][parts * n][k], codes with their blocks' scales or tokens, as fp32."""
    if s is None:
        return w.float()
    n, k = w.shape[-2] // parts, w.shape[-1]
    lead = w.shape[:-2]
    s = _spread(s.reshape(*lead, parts, _groups(n), _groups(k)), -2, n)
    return (w.float().view(*lead, parts, n, k) * _spread(s, -1, k)).view(w.shape)


def _code(v, kind, group):
    """Codes and scales of fp32 values [..][k] in groups of `group` elements (the last may be short)."""
    k = v.shape[-1]
    p = torch.nn.functional.pad(v.abs(), (0, -k % group))
    amax = p.view(*v.shape[:-1], -1, group).amax(-1)
    dyn = torch.where(amax > 0, _TOP[kind] / amax, 0.0)
    codes = (v * dyn.repeat_interleave(group, -1)[..., :k]).clamp(-_TOP[kind], _TOP[kind])
    return codes.to(_CODE[kind]), torch.where(amax > 0, 1.0 / dyn, 0.0)


def _decode(codes, scales, token):
    """What codes with a scale per 128 columns stand for, in the token type."""
    rows, k = codes.shape
    if k % _BLOCK:
        return (codes.float() * _spread(scales, 1, k)).to(token)
    codes = codes.to(token).view(rows, -1, _BLOCK)         # exact
    return torch.mul(codes, scales[:, :, None], out=torch.empty_like(codes)).view(rows, k)


def _swiglu(y, dim):
    gate, up = y.chunk(2, dim)
    return gate / (1.0 + torch.exp(-gate)) * up


def _plain_block(st):
    """The rows of all experts side by side, padded to the longest, in one batched product."""
    case = st["case"]
    rows, din = st["x"].shape
    at = st["first"][:, None] + torch.arange(st["most"], device=st["x"].device)
    here = torch.arange(st["most"], device=st["x"].device) < st["many"][:, None]
    x = st["x"].float() * _spread(st["xs"], 1, din)
    x = x[at.clamp(max=rows - 1)].transpose(1, 2).contiguous()
    y = torch.bmm(_values(st["w"], st["ws"], 2 if case["swiglu"] else 1), x)
    if case["swiglu"]:
        y = _swiglu(y, 1)
    y = y.transpose(1, 2)[here]
    if case["codes"]:
        return _decode(*_code(y, case["codes"], _BLOCK), torch.bfloat16)
    return y.to(torch.bfloat16)


def _plain_norm(st):
    case = st["case"]
    s, out = st["x"].float(), {}
    if st["residual"] is not None:
        s = s + st["residual"].float()
        out["residual_out"] = s.to(st["x"].dtype)
    y = s * torch.rsqrt((s * s).mean(2, keepdim=True) + 1e-6) * st["gamma"].float()
    out["y"] = y.to(st["x"].dtype)
    if case["mode"]:
        out["codes"], scales = _code(y, case["codes"], case["H"] if case["mode"] == 2 else _BLOCK)
        out["dynamic_scales"] = scales.view(case["W"] * case["BS"], -1)
    return out


def _plain_few(st):
    """Each pick's own copy of its expert's weights, in one batched product."""
    case, ids = st["case"], st["ids"].flatten()
    T, K, H = case["W"] * case["BS"], case["K"], case["H"]
    bits = lambda w, s: (w if s is None else w.view(torch.uint8))[ids].view(w.dtype)  # noqa: E731
    x = st["x"].float().view(T, 1, H).expand(T, K, H).reshape(T * K, H, 1)
    up = _values(bits(st["up"], st["ups"]), None if st["ups"] is None else st["ups"][ids], 2)
    h = _swiglu(torch.bmm(up, x), 1)
    del up
    down = _values(bits(st["down"], st["downs"]), None if st["downs"] is None else st["downs"][ids], 1)
    o = torch.bmm(down, h).view(T, K, H)
    weight = st["weight"].view(T, K, 1)
    if st["mask"] is not None:
        weight = weight * st["mask"].view(T, 1, 1)
    return (o * weight).sum(1).to(st["x"].dtype).view(st["x"].shape)


def run(state):
    case = state["case"]
    if not own:
        return {"block": _plain_block, "codes": _plain_block, "norm": _plain_norm,
                "few": _plain_few}[case["op"]](state)
    state["launch"]()
    if case["op"] == "codes":
        codes, scales = state["out"]
        return _decode(codes.view(_CODE[case["codes"]]), scales, torch.bfloat16)
    if case["op"] != "norm":
        return state["out"]
    out = {k: v for k, v in state["out"].items() if v is not None}
    if case["mode"]:
        out["codes"] = out["codes"].view(_CODE[case["codes"]])
        out["dynamic_scales"] = out["dynamic_scales"].view(case["W"] * case["BS"], -1)
    return out


# -- what a pass cannot do without ----------------------------------------------------------

def _expected_active(E, K, T):
    """Experts expected to have rows: their weights have to be read."""
    return E * (1.0 - (1.0 - K / E) ** T)


def work(case):
    if case["op"] == "norm":
        n = case["W"] * case["BS"] * case["H"]
        each = 2 + (4 if case["residual"] else 0) + 2 + (1 if case["mode"] else 0)
        scales = {0: 0, 2: 1, 3: _groups(case["H"])}[case["mode"]] * case["W"] * case["BS"] * 4
        return {"bytes": n * each + case["H"] * 2 + scales, "flops": 8 * n}
    if case["op"] == "few":
        E, K, H, F, T = case["E"], case["K"], case["H"], case["F"], case["active"]
        size = 2.0 if case["weights"] == "token" else 1.0 + 4.0 / _BLOCK ** 2
        return {"bytes": int(_expected_active(E, K, T) * 3 * H * F * size + 4 * T * H + 8 * T * K),
                "flops": 6 * T * K * H * F}
    rows, din, dout = case["W"] * case["BS"] * case["K"], case["din"], case["dout"]
    cols = dout // 2 if case["swiglu"] else dout
    out = rows * (cols + 4 * _groups(cols)) if case["codes"] else rows * cols * 2
    active = _expected_active(case["E"], case["K"], case["W"] * case["BS"])
    return {"bytes": int(rows * (din + 4 * _groups(din)) + active * dout * din * (1 + 4 / _BLOCK ** 2) + out),
            "flops": 2 * rows * din * dout}


# -- the definition in 64 bits ----------------------------------------------------------------

def _exact_weight(w, s, parts):
    """One expert's weights: every element times the scale of its block, block by block row."""
    v = w.double()
    if s is None:
        return v
    n = v.shape[0] // parts
    row = torch.arange(v.shape[0], device=v.device)
    block = torch.div(row % n, _BLOCK, rounding_mode="floor") + torch.div(row, n, rounding_mode="floor") * _groups(n)
    col = torch.div(torch.arange(v.shape[1], device=v.device), _BLOCK, rounding_mode="floor")
    return v * s.double()[block][:, col]


def _exact_code(v, kind):
    """The values of the code type next to fp64 values, ties to even."""
    bits, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[kind]
    step = torch.ldexp(torch.ones_like(v), torch.frexp(v).exponent.clamp(min=least + 1) - 1 - bits)
    return (torch.round(v / step) * step).clamp(-_TOP[kind], _TOP[kind])


def _exact_gated(v):
    half = v.shape[1] // 2
    return v[:, :half] * torch.sigmoid(v[:, :half]) * v[:, half:]


def _exact_block(case, st):
    col = torch.div(torch.arange(case["din"], device=_DEV), _BLOCK, rounding_mode="floor")
    done = []
    for e, (lo, n) in enumerate(zip(st["first"].tolist(), st["many"].tolist())):
        x = st["x"][lo:lo + n].double() * st["xs"][lo:lo + n].double()[:, col]
        v = x @ _exact_weight(st["w"][e], st["ws"][e], 2 if case["swiglu"] else 1).t()
        done.append(_exact_gated(v) if case["swiglu"] else v)
    y = torch.cat(done)
    if case["codes"]:
        scales = [p.abs().amax(1, keepdim=True) / _TOP[case["codes"]] for p in y.split(_BLOCK, 1)]
        y = torch.cat([_exact_code(p / v, case["codes"]) * v for p, v in zip(y.split(_BLOCK, 1), scales)], 1)
    return y


def _exact_norm(case, st):
    s = st["x"].double()
    out = {}
    if st["residual"] is not None:
        s = s + st["residual"].double()
        out["residual_out"] = s
    y = s / torch.sqrt(torch.mean(s ** 2, 2, keepdim=True) + 1e-6) * st["gamma"].double()
    out["y"] = y
    if case["mode"]:
        parts = y.view(-1, case["H"]).split(case["H"] if case["mode"] == 2 else _BLOCK, 1)
        scales = [p.abs().amax(1, keepdim=True) / _TOP[case["codes"]] for p in parts]
        out["codes"] = torch.cat([_exact_code(p / v, case["codes"]) for p, v in zip(parts, scales)], 1).view(y.shape)
        out["dynamic_scales"] = torch.cat(scales, 1)
    return out


def _exact_few(case, st):
    T, K, H = case["W"] * case["BS"], case["K"], case["H"]
    ids, weight = st["ids"].view(T, K).long(), st["weight"].view(T, K).double()
    if st["mask"] is not None:
        ids = torch.where(st["mask"].view(T, 1), ids, -1)
    x = st["x"].view(T, H).double()
    y = torch.zeros((T, H), dtype=torch.float64, device=_DEV)
    for e in range(case["E"]):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        up = _exact_weight(st["up"][e], None if st["ups"] is None else st["ups"][e], 2)
        down = _exact_weight(st["down"][e], None if st["downs"] is None else st["downs"][e], 1)
        y.index_add_(0, t, (_exact_gated(x[t] @ up.t()) @ down.t()) * weight[t, k][:, None])
    return y.view(st["x"].shape)


def exact(case, seed):
    global own
    mine, own = own, False           # the inputs alone
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    return {"block": _exact_block, "codes": _exact_block, "norm": _exact_norm,
            "few": _exact_few}[case["op"]](case, st)
