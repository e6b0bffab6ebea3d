"""Measured cases of the 8-bit floating point operators: activations quantised by blocks of
128 inputs, the block-scaled linear layer, routing to experts and the experts' gated products.

Definitions (all sums, scales and scores in 32 bits or more):

  quantise   v = x, or silu(gate) * up for a gated row [gate | up];  per row and block of 128
             consecutive inputs (the last one may be shorter):
             a = max(max |v|, 2^-100),  q = e4m3(fl32(v * fl32(448 / a))),  scale = fl32(a / 448).
             Scales come block by block: [ceil(K / 128), M].
  linear     y[m, n] = sum_b scale_x[b, m] scale_w[n / 128, b] sum_{k in b} q[m, k] w[n, k]
             with x quantised as above and w e4m3 codes [N, K], one scale per 128 x 128 block.
  route      scores p = softmax(logits) or sigmoid(logits); an expert is chosen by its score
             plus a bias; groups of experts rank by their best expert (softmax) or the sum of
             their best two (sigmoid) and only the best groups stay; the k best experts in
             falling order, ties to the lowest index. Weights are the scores without the bias,
             renormalised to sum 1 if asked, times a factor. An expert at -inf or NaN is never
             chosen; a slot that nothing is left for holds index -1 and weight 0.
  experts    y[m] = sum_j weight[m, j] * linear(quantise([x Wg^T | x Wu^T], gated), Wd) with
             the matrices of expert index[m, j]; slots at -1 add nothing.
"""
import math

import torch

own = False

DEV = "cuda"
HALF = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
FLOOR = 2.0 ** -100


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode batch's inputs to a 70B-shaped projection
        {"name": "quant 16x8192", "op": "quant", "M": 16, "K": 8192, "gated": False, "dtype": "fp16"},
        # 3B-shaped gate|up outputs of a prefill batch: 8640 inputs end inside a block of 128
        {"name": "quant gated 2048x8640", "op": "quant", "M": 2048, "K": 8640, "gated": True, "dtype": "bf16"},
        # one token through a 70B-shaped square projection
        {"name": "linear 1x8192x8192", "op": "linear", "M": 1, "N": 8192, "K": 8192, "dtype": "fp16", "out": "fp32"},
        # a decode batch through the 70B-shaped gate projection
        {"name": "linear 16x28672x8192", "op": "linear", "M": 16, "N": 28672, "K": 8192, "dtype": "bf16", "out": "bf16"},
        # 3B-shaped down projection of a prefill of 512 tokens (ragged K, N = 25 blocks)
        {"name": "linear 512x3200x8640", "op": "linear", "M": 512, "N": 3200, "K": 8640, "dtype": "fp16", "out": "fp32"},
        # a long prefill through the 70B-shaped gate projection
        {"name": "linear 4096x28672x8192", "op": "linear", "M": 4096, "N": 28672, "K": 8192, "dtype": "bf16", "out": "bf16"},
        # one token's routing, sigmoid scores with a balance bias and groups
        {"name": "route 1x256 sigmoid", "op": "route", "M": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "renorm": True, "factor": 2.5, "masked": 0.0, "dtype": "fp32"},
        # a long prefill's routing over the same experts
        {"name": "route 16384x256 sigmoid", "op": "route", "M": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "renorm": True, "factor": 2.5, "masked": 0.0, "dtype": "fp32"},
        # softmax scores without groups, bf16 logits, some experts masked out
        {"name": "route 4096x60 softmax", "op": "route", "M": 4096, "E": 60, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "kept": 1, "renorm": False, "factor": 1.0, "masked": 0.1, "dtype": "bf16"},
        # one token through its eight experts
        {"name": "experts 1 of 64", "op": "experts", "M": 1, "E": 64, "k": 8, "H": 4096, "I": 1024, "held": 1.0, "dtype": "bf16"},
        # a decode batch that reaches nearly every expert; inner width ends inside a block
        {"name": "experts 48 of 64", "op": "experts", "M": 48, "E": 64, "k": 8, "H": 4096, "I": 1104, "held": 1.0, "dtype": "fp16"},
        # a long prefill
        {"name": "experts 4096 of 64", "op": "experts", "M": 4096, "E": 64, "k": 8, "H": 4096, "I": 1024, "held": 1.0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "route", "experts"])
    if op == "quant":
        M = _log(rng, 1, 4096)
        K = 16 * _log(rng, 1, min(28672, 2048 * 8640 * 2 // M) // 16)
        return {"op": op, "M": M, "K": K, "gated": rng.random() < 0.5, "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    if op == "linear":
        M = _log(rng, 1, 4096)
        N, K = _log(rng, 64, 28672), 16 * _log(rng, 8, 1792)
        while N * K > 28672 * 8192:
            N, K = _log(rng, 64, 28672), 16 * _log(rng, 8, 1792)
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["fp16", "bf16", "fp32"]), "out": rng.choice(["fp16", "bf16", "fp32"])}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, 8 // groups), 512 // groups)
        kept = rng.randint((groups + 1) // 2, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "M": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E // groups * kept)), "score": score,
                "bias": score == "sigmoid" and rng.random() < 0.7, "groups": groups, "kept": kept, "renorm": rng.random() < 0.5,
                "factor": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.1, 0.9]), "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    E = rng.randint(4, 64)
    M = _log(rng, 1, 4096)
    return {"op": op, "M": M, "E": E, "k": rng.randint(1, min(8, E)), "H": 16 * _log(rng, 32, 256),
            "I": 16 * _log(rng, 8, 64), "held": rng.choice([1.0, 1.0, 0.25]) if M > 15 else 1.0, "dtype": rng.choice(["fp16", "bf16"])}


def work(case):
    c, two = case, {"fp16": 2, "bf16": 2, "fp32": 4}
    if c["op"] == "quant":
        n = c["M"] * c["K"]
        return {"bytes": n * two[c["dtype"]] * (2 if c["gated"] else 1) + n + 4 * c["M"] * -(-c["K"] // 128), "flops": 0}
    if c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": M * K * two[c["dtype"]] + N * K + 4 * -(-N // 128) * -(-K // 128) + M * N * two[c["out"]], "flops": 2 * M * N * K}
    if c["op"] == "route":
        return {"bytes": c["M"] * (c["E"] * two[c["dtype"]] + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0), "flops": 0}
    M, E, k, H, I = c["M"], c["E"], c["k"], c["H"], c["I"]
    pairs = M * k * c["held"]
    reached = E * (1 - (1 - 1 / E) ** pairs) if M > 1 else min(E, pairs)  # experts with at least one token, of which each is read once
    return {"bytes": int(reached * 3 * H * I + 2 * M * H * two[c["dtype"]] + 8 * M * k), "flops": int(6 * pairs * H * I)}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _gen(seed, at):
    return torch.Generator(device=DEV).manual_seed(seed * 16 + at)


def _activations(shape, dtype, seed, at):
    """Hidden states: normal values, with a few channels ten times larger than the rest."""
    x = torch.randn(shape, generator=_gen(seed, at), device=DEV)
    loud = torch.rand(shape[-1], generator=_gen(seed, at + 1), device=DEV) < 0.005
    return torch.where(loud, 10 * x, x).to(HALF[dtype])


def _weights(shape, seed, at):
    """e4m3 codes [..., N, K] of normal weights and their scales [..., ceil(N / 128), ceil(K / 128)]."""
    *lead, N, K = shape
    nb, kb = -(-N // 128), -(-K // 128)
    w = torch.zeros(*lead, nb * 128, kb * 128, device=DEV)
    w[..., :N, :K] = torch.randn(*lead, N, K, generator=_gen(seed, at), device=DEV) * (K ** -0.5)
    blocks = w.view(*lead, nb, 128, kb, 128)
    scale = blocks.abs().amax((-3, -1)).clamp_min(FLOOR) / 448.0
    codes = (blocks / scale[..., :, None, :, None]).clamp(-448, 448).view(*lead, nb * 128, kb * 128)[..., :N, :K]
    return codes.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


def prepare(case, seed):
    c, s = case, {"case": dict(case)}
    if c["op"] in ("quant", "linear"):
        s["x"] = _activations((c["M"], c["K"] * (2 if c.get("gated") else 1)), c["dtype"], seed, 0)
        if c["op"] == "linear":
            s["w"], s["sw"] = _weights((c["N"], c["K"]), seed, 2)
    elif c["op"] == "route":
        popular = torch.randn(c["E"], generator=_gen(seed, 0), device=DEV) * 0.5
        l = torch.randn(c["M"], c["E"], generator=_gen(seed, 1), device=DEV) + popular
        gone = torch.rand(c["M"], c["E"], generator=_gen(seed, 2), device=DEV) < c["masked"]
        s["logits"] = torch.where(gone, -math.inf, l).to(HALF[c["dtype"]])
        # a balance bias moves by steps of 0.001 during training
        s["bias"] = torch.round(torch.randn(c["E"], generator=_gen(seed, 3), device=DEV) * 20) * 0.001 if c["bias"] else None
    else:
        E, H, I = c["E"], c["H"], c["I"]
        s["x"] = _activations((c["M"], H), c["dtype"], seed, 0)
        s["wgu"], s["sgu"] = _weights((E, 2, I, H), seed, 2)
        s["wd"], s["sd"] = _weights((E, H, I), seed, 3)
        popular = torch.randn(E, generator=_gen(seed, 4), device=DEV) * 0.3
        l = torch.randn(c["M"], E, generator=_gen(seed, 5), device=DEV) + popular
        p, idx = torch.topk(torch.softmax(l, 1), c["k"], 1)
        away = torch.rand(c["M"], c["k"], generator=_gen(seed, 6), device=DEV) >= c["held"]  # slots that another rank's experts serve
        s["index"] = torch.where(away, -1, idx).to(torch.int32)
        s["weight"] = (p / p.sum(1, keepdim=True)).contiguous()
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def _quantise(v):
    M, K = v.shape
    kb = -(-K // 128)
    b = torch.nn.functional.pad(v, (0, kb * 128 - K)).view(M, kb, 128)
    a = b.abs().amax(2).clamp_min(FLOOR)
    q = (b * (448.0 / a)[:, :, None]).to(torch.float8_e4m3fn).view(M, kb * 128)[:, :K]
    return q.contiguous(), (a / 448.0).t().contiguous()


def _gate(v):
    g, u = v.chunk(2, 1)
    return g / (1 + torch.exp(-g)) * u


def _values(codes, scale, rows):
    """e4m3 codes [M, K] with scales [ceil(M / rows), ceil(K / 128)] as 32-bit values."""
    M, K = codes.shape
    return codes.float() * scale.repeat_interleave(rows, 0)[:M].repeat_interleave(128, 1)[:, :K]


def _linear(v, w, sw):
    q, s = _quantise(v)
    return _values(q, s.t(), 1) @ _values(w, sw, 128).t()


def _route(l, c, bias):
    M, E = l.shape
    l = l.float()
    ok = l > -math.inf
    l = torch.where(ok, l.clamp_max(torch.finfo(torch.float32).max), -math.inf)
    if c["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-l))
        choice = p if bias is None else p + bias
    else:
        e = torch.where(ok, torch.exp(l - l.amax(1, keepdim=True)), 0)
        p = e / e.sum(1, keepdim=True)
        choice = l if bias is None else p + bias  # a softmax keeps the logits' order
    choice = torch.where(ok & (choice > -math.inf), choice, -math.inf)
    if c["groups"] > 1:
        in_group = choice.view(M, c["groups"], -1)
        best = in_group.sort(dim=2, descending=True)[0][:, :, :2]
        if c["score"] == "sigmoid":
            rank = best[:, :, 0] + torch.where(best[:, :, -1] > -math.inf, best[:, :, -1], 0) * (best.shape[2] - 1)
        else:
            rank = best[:, :, 0]
        keep = rank.sort(dim=1, descending=True, stable=True)[1][:, : c["kept"]]
        mask = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, keep, True)
        choice = torch.where(mask[:, :, None], in_group, -math.inf).view(M, E)
    order = choice.sort(dim=1, descending=True, stable=True)[1][:, : c["k"]]
    taken = choice.gather(1, order) > -math.inf
    weight = torch.where(taken, p.gather(1, order), 0)
    if c["renorm"]:
        total = weight.sum(1, keepdim=True)
        weight = torch.where(total > 0, weight / total, 0)
    return {"weight": weight * c["factor"], "index": torch.where(taken, order, -1).to(torch.int32)}


def _experts(s):
    x, index, weight = s["x"].float(), s["index"], s["weight"]
    y = torch.zeros_like(x)
    for e in index.unique().tolist():  # each expert multiplies the tokens that chose it
        if e < 0:
            continue
        token, slot = torch.nonzero(index == e, as_tuple=True)
        v = torch.cat([_linear(x[token], s["wgu"][e, i], s["sgu"][e, i]) for i in (0, 1)], 1)
        y.index_add_(0, token, _linear(_gate(v), s["wd"][e], s["sd"][e]) * weight[token, slot, None])
    return y.to(s["x"].dtype)


def _own(s):
    import ternary_weight_linear_amd as tw

    c = s["case"]
    if c["op"] == "quant":
        q, scale = tw.bl_quant_act_fp8(s["x"], gated=c["gated"])
        return {"q": q, "scale": scale}
    if c["op"] == "linear":
        return tw.bl_fp8_forward(s["x"], s["w"], s["sw"], out_dtype=HALF[c["out"]])
    if c["op"] == "route":
        weight, index = tw.bl_route_experts(s["logits"], c["k"], bias=s["bias"], score=c["score"], groups=c["groups"], kept_groups=c["kept"],
                                            renorm=c["renorm"], factor=c["factor"])
        return {"weight": weight, "index": index}
    return tw.bl_fp8_experts(s["x"], s["index"], s["weight"], s["wgu"], s["sgu"], s["wd"], s["sd"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "quant":
        v = state["x"].float()
        q, scale = _quantise(_gate(v) if c["gated"] else v)
        return {"q": q, "scale": scale}
    if c["op"] == "linear":
        return _linear(state["x"].float(), state["w"], state["sw"]).to(HALF[c["out"]])
    if c["op"] == "route":
        return _route(state["logits"], c, state["bias"])
    return _experts(state)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _e4m3(t):
    """The nearest e4m3 value (ties to even) of each |t| <= 448(1 + 2^-20), in 64 bits."""
    unit = torch.exp2(torch.frexp(t)[1].clamp_min(-5).double() - 4)  # 4 bits of mantissa, least unit 2^-9
    return torch.round(t / unit) * unit


def _quantised64(v):
    """(codes, scales [M, ceil(K / 128)]) of 64-bit values; codes are decided in 32 bits, as the definition says."""
    M, K = v.shape
    parts = []
    for at in range(0, K, 128):
        b = v[:, at:at + 128]
        a = b.abs().max(1, keepdim=True)[0].clamp(min=FLOOR)
        r = (448 / a.float()).double()
        parts.append((_e4m3((b.float().double() * r).float().double()), a / 448))
    return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts], 1)


def _times64(v, w, sw):
    codes, scale = _quantised64(v)
    y = torch.zeros(v.shape[0], w.shape[0], dtype=torch.float64, device=v.device)
    wide = 16  # blocks of inputs that are spread out at a time
    for b in range(0, scale.shape[1], wide):
        at = slice(b * 128, min((b + wide) * 128, v.shape[1]))
        block = torch.arange(at.start, at.stop, device=v.device) // 128
        row = torch.arange(w.shape[0], device=v.device) // 128
        y += (codes[:, at] * scale[:, block]) @ (w[:, at].double() * sw.double()[row][:, block]).t()
    return y


def _silu64(g, u):
    return g * torch.sigmoid(g) * u


def _route64(s, c):
    l = s["logits"].double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    choice = (p if c["score"] == "sigmoid" else l) if s["bias"] is None else p + s["bias"].double()
    choice = choice.masked_fill(l == -math.inf, -math.inf)
    M, E = l.shape
    size = E // c["groups"]
    if c["groups"] > 1:
        grouped = choice.reshape(M, c["groups"], size)
        first = torch.topk(grouped, min(2, size), 2)[0]
        rank = first[..., 0].clone()
        if c["score"] == "sigmoid" and size > 1:
            rank += first[..., 1].masked_fill(first[..., 1] == -math.inf, 0)
        worse = torch.argsort(torch.argsort(-rank, dim=1, stable=True), dim=1) >= c["kept"]
        choice = grouped.masked_fill(worse[..., None], -math.inf).reshape(M, E)
    at = torch.argsort(-choice, dim=1, stable=True)[:, : c["k"]]
    w = torch.gather(p, 1, at) * (torch.gather(choice, 1, at) > -math.inf)
    if c["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    return w * c["factor"]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "quant":
        v = s["x"].double()
        codes, scale = _quantised64(_silu64(v[:, : c["K"]], v[:, c["K"]:]) if c["gated"] else v)
        return {"q": codes, "scale": scale.t().contiguous()}
    if c["op"] == "linear":
        return _times64(s["x"].double(), s["w"], s["sw"])
    if c["op"] == "route":
        return {"weight": _route64(s, c), "index": None}
    x, y = s["x"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        chosen = (s["index"] == e)
        rows = chosen.any(1).nonzero()[:, 0]
        if rows.numel():
            g, u = (_times64(x[rows], s["wgu"][e, i], s["sgu"][e, i]) for i in (0, 1))
            w = (s["weight"].double() * chosen).sum(1)[rows]
            y[rows] += w[:, None] * _times64(_silu64(g, u), s["wd"][e], s["sd"][e])
    return y
