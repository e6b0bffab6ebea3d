"""Measured cases of what is trained around frozen weights: low-rank adapters of many requests
beside a shared projection with their gradients, the experts' balance loss with its counts, and
the gradient of the router's logits.

Definitions (all sums, scores and statistics in 32 bits or more; e = index[m] where it names one
of the L adapters, whose matrices are a[e] [R, K] and, transposed, b[e] [R, N], scaled by s[e]):

  adapters   h[m, r] = sum_k a[e, r, k] x[m, k],   y[m, n] = base[m, n] + s[e] sum_r b[e, r, n] h[m, r];
             a row without an adapter keeps its base and has h = 0.
  adapter gradients
             dh[m, r] = s[e] sum_n b[e, r, n] dy[m, n],   dx[m, k] = base[m, k] + sum_r a[e, r, k] dh[m, r],
             da[e, r, k] = sum_m dh[m, r] x[m, k],   db[e, r, n] = s[e] sum_m h[m, r] dy[m, n],
             the last two over the adapter's rows (zeros where it has none).
  balance    Scores p = softmax(logits) or sigmoid(logits), t[m, e] = p[m, e] / sum_e p[m, e]; an
             expert at -inf has none. Over the rows m of one sequence that chose any expert, of
             which there are T, with count[e] slots of each expert and C slots in all:
             coef[e] = E count[e] / (C T),   loss = sum_e coef[e] sum_m t[m, e].
             Rows of no sequence count nowhere.
  router gradient
             Routing weights w[m, j] = factor p[m, index[m, j]], divided by their row's sum of p if
             renormalised. dlogits = the gradient of sum w dweight + sum over sequences dloss loss,
             with the counts held fixed.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # one token of one request beside a 70B-shaped square projection, whose outputs are fp32
        {"name": "adapters 1x8192x8192", "op": "adapters", "M": 1, "K": 8192, "N": 8192, "L": 64, "R": 16, "mix": "rows", "bare": 0.0,
         "dtype": "fp16", "out": "fp32"},
        # a decode batch of requests that mostly have an adapter of their own, beside a 70B-shaped gate projection
        {"name": "adapters 48x28672x8192", "op": "adapters", "M": 48, "K": 8192, "N": 28672, "L": 64, "R": 16, "mix": "rows", "bare": 0.1,
         "dtype": "bf16", "out": "bf16"},
        # a wide decode batch of requests that share few adapters
        {"name": "adapters 320x4096x4096", "op": "adapters", "M": 320, "K": 4096, "N": 4096, "L": 12, "R": 32, "mix": "rows", "bare": 0.2,
         "dtype": "bf16", "out": "fp32"},
        # prompts of some requests beside a 3B-shaped down projection, ranks that fill no tile
        {"name": "adapters 777x3200x8640", "op": "adapters", "M": 777, "K": 8640, "N": 3200, "L": 5, "R": 12, "mix": "runs", "bare": 0.1,
         "dtype": "fp16", "out": "fp32"},
        # long prompts of eight requests beside a 70B-shaped square projection
        {"name": "adapters 4096x8192x8192", "op": "adapters", "M": 4096, "K": 8192, "N": 8192, "L": 8, "R": 64, "mix": "runs", "bare": 0.0,
         "dtype": "bf16", "out": "bf16"},
        # a small training step in fp32 with sizes that are no multiple of anything
        {"name": "adapter gradients 301x777x1001", "op": "adapter_grad", "M": 301, "K": 1001, "N": 777, "L": 3, "R": 5, "mix": "runs", "bare": 0.1,
         "dtype": "fp32", "out": "fp32"},
        # a step on three packed fine-tunings of a 3B-shaped gate projection whose gradients arrive in fp32
        {"name": "adapter gradients 1024x8640x3200", "op": "adapter_grad", "M": 1024, "K": 3200, "N": 8640, "L": 3, "R": 8, "mix": "runs", "bare": 0.0,
         "dtype": "fp16", "out": "fp32"},
        # a step of one fine-tuning on a long batch, 70B-shaped square projection
        {"name": "adapter gradients 4096x8192x8192", "op": "adapter_grad", "M": 4096, "K": 8192, "N": 8192, "L": 1, "R": 32, "mix": "runs", "bare": 0.0,
         "dtype": "bf16", "out": "bf16"},
        # the loss of a batch's routing as one sequence, bf16 logits, some experts masked out
        {"name": "balance 4096x60 softmax", "op": "balance", "M": 4096, "E": 60, "k": 4, "S": 1, "score": "softmax", "masked": 0.1, "dtype": "bf16"},
        # the loss per packed sequence of a long batch with rows behind the last one
        {"name": "balance 16384x256 sigmoid", "op": "balance", "M": 16384, "E": 256, "k": 8, "S": 11, "score": "sigmoid", "masked": 0.0, "dtype": "fp32"},
        # the router's gradient in the same two batches
        {"name": "router gradient 4096x60 softmax", "op": "route_grad", "M": 4096, "E": 60, "k": 4, "S": 1, "score": "softmax", "masked": 0.1,
         "renorm": False, "factor": 1.0, "dtype": "bf16"},
        {"name": "router gradient 16384x256 sigmoid", "op": "route_grad", "M": 16384, "E": 256, "k": 8, "S": 11, "score": "sigmoid", "masked": 0.0,
         "renorm": True, "factor": 2.5, "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adapters", "adapters", "adapters", "adapter_grad", "adapter_grad", "balance", "route_grad"])
    if op in ("adapters", "adapter_grad"):
        most = 4096 * 16384 * (64 if op == "adapters" else 32)
        while True:
            M, L, R = _log(rng, 1, 4096), _log(rng, 1, 64), _log(rng, 2, 64)
            # widths of models are multiples of 8 or more, seldom anything else
            unit = rng.choice([1, 8, 16, 64, 64])
            K, N = (unit * max(1, _log(rng, 64, 28672) // unit) for _ in range(2))
            if M * (K + N) * R <= most and M * (K + N) <= 4096 * 16384 and L * R * (K + N) <= 1 << 27:
                break
        dtype = rng.choice(["fp16", "bf16", "bf16", "fp32"])
        return {"op": op, "M": M, "K": K, "N": N, "L": L, "R": R, "mix": "rows" if op == "adapters" and M <= 512 and rng.random() < 0.6 else "runs",
                "bare": rng.choice([0.0, 0.1, 0.5]) if M > 8 else 0.0, "dtype": dtype, "out": rng.choice([dtype, "fp32"])}
    E = _log(rng, 4, 512)
    M = _log(rng, 1, 16384 if E <= 256 else 8192)
    c = {"op": op, "M": M, "E": E, "k": rng.randint(1, min(8, E)), "S": _log(rng, 1, min(M, 32)), "score": rng.choice(["softmax", "sigmoid"]),
         "masked": rng.choice([0.0, 0.0, 0.1, 0.9]), "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    return c if op == "balance" else {**c, "renorm": rng.random() < 0.5, "factor": rng.choice([1.0, 2.5])}


def work(case):
    c = case
    M, size = c["M"], BYTES[c["dtype"]]
    if c["op"] in ("adapters", "adapter_grad"):
        K, N, L, R, out = c["K"], c["N"], c["L"], c["R"], BYTES[c["out"]]
        used = M * (1 - c["bare"])
        reached = min(L, used) if c["mix"] == "runs" else L * (1 - (1 - 1 / L) ** used)  # adapters of any row, read once each
        bytes_ = reached * R * (K + N) * size + M * K * size + 4 * M * R + 4 * M + 4 * L
        if c["op"] == "adapters":
            return {"bytes": int(bytes_ + 2 * M * N * out), "flops": int(2 * used * R * (K + N))}
        return {"bytes": int(bytes_ + M * N * out + 2 * M * K * out + 4 * L * R * (K + N)), "flops": int(4 * used * R * (K + N))}
    E, k, S = c["E"], c["k"], c["S"]
    if c["op"] == "balance":
        return {"bytes": M * (E * size + 4 * k) + 8 * S * E + 8 * S, "flops": 0}
    return {"bytes": M * (2 * E * size + 8 * k) + 4 * S * E + 8 * S, "flops": 0}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------
def _gen(seed, at):
    return torch.Generator(device=DEV).manual_seed(seed * 32 + at)


def _randn(shape, seed, at):
    return torch.randn(shape, generator=_gen(seed, at), device=DEV)


def _rand(shape, seed, at):
    return torch.rand(shape, generator=_gen(seed, at), device=DEV)


def _activations(shape, dtype, seed, at):
    """Hidden states: normal values, with a few channels ten times larger than the rest."""
    x = _randn(shape, seed, at)
    loud = _rand(shape[-1], seed, at + 1) < 0.005
    return torch.where(loud, 10 * x, x).to(TYPES[dtype])


def _runs(M, count, seed, at):
    """Offsets int32 [count + 1] of count packed sequences of random lengths over M rows."""
    inner = torch.floor(_rand(count - 1, seed, at) * M).sort()[0]
    return torch.cat([torch.zeros(1, device=DEV), inner, torch.full((1,), float(M), device=DEV)]).to(torch.int32)


def _row_sequence(M, offsets):
    """The sequence of each row, int64 [M] (rows behind the last one: their count)."""
    return torch.searchsorted(offsets[1:].contiguous(), torch.arange(M, device=DEV, dtype=torch.int32), right=True)


def _prepare_adapters(c, seed):
    M, K, N, L, R = (c[n] for n in "MKNLR")
    dtype, out = TYPES[c["dtype"]], TYPES[c["out"]]
    s = {"x": _activations((M, K), c["dtype"], seed, 0)}
    s["a"] = (_randn((L, R, K), seed, 2) * K ** -0.5).to(dtype)
    s["b"] = (_randn((L, R, N), seed, 3) * R ** -0.5).to(dtype)
    s["scale"] = 0.25 * 2.0 ** torch.floor(4 * _rand(L, seed, 4))
    if c["mix"] == "rows":
        e = torch.floor(_rand(M, seed, 5) * L)
    else:  # requests one after another; each has its adapter, two may have the same
        count = min(M, L + L // 2)
        e = torch.floor(_rand(count, seed, 5) * L)
        e[: min(L, count)] = torch.randperm(L, generator=_gen(seed, 6), device=DEV)[:count].float()
        e = e[_row_sequence(M, _runs(M, count, seed, 7)).clamp_max(count - 1)]
    s["index"] = torch.where(_rand(M, seed, 8) < c["bare"], -1, e).to(torch.int32)
    if c["op"] == "adapters":
        s["base"] = _randn((M, N), seed, 9).to(out)
        return s
    s["dy"] = _randn((M, N), seed, 10).to(out)
    s["base"] = _randn((M, K), seed, 11).to(out)
    s["h"] = _spread(s["x"].float() @ s["a"].float().flatten(0, 1).t(), s["index"], L)[0]  # the forward pass left it
    return s


def _prepare_route(c, seed):
    M, E, k, S = c["M"], c["E"], c["k"], c["S"]
    popular = _randn(E, seed, 0) * 0.5
    l = _randn((M, E), seed, 1) + popular
    s = {"logits": torch.where(_rand((M, E), seed, 2) < c["masked"], -math.inf, l).to(TYPES[c["dtype"]])}
    top, index = s["logits"].float().topk(k, 1)
    s["index"] = torch.where(top > -math.inf, index, -1).to(torch.int32)
    s["offsets"] = _runs(M, S, seed, 3) if S > 1 else None
    if S > 2:
        s["offsets"][-1] = s["offsets"][-2]  # the last sequence is empty, and its rows belong to none
    if c["op"] == "route_grad":
        s["dweight"] = _randn((M, k), seed, 4)
        s["dloss"] = 0.5 + _rand(S, seed, 5)
        count, rows = _counts(s["index"], E, _of_rows(c, s), S)
        s["coef"] = _coef(count, rows)  # the loss left it
    return s


def _of_rows(c, s):
    return torch.zeros(c["M"], dtype=torch.int64, device=DEV) if s["offsets"] is None else _row_sequence(c["M"], s["offsets"])


def prepare(case, seed):
    s = _prepare_adapters(case, seed) if case["op"] in ("adapters", "adapter_grad") else _prepare_route(case, seed)
    return {"case": dict(case), **s}


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------
def _spread(all_, index, L):
    """Of [M, L R] values of every adapter: each row's own, [M, R], and the rest as zeros, [M, L R]."""
    M = index.shape[0]
    mine = (index[:, None] == torch.arange(L, device=DEV)).float()
    kept = all_.view(M, L, -1) * mine[:, :, None]
    return kept.sum(1), kept.view(M, -1)


def _place(h, index, L):
    """[M, R] values at their adapter's place in [M, L R]."""
    mine = (index[:, None] == torch.arange(L, device=DEV)).float()
    return (mine[:, :, None] * h[:, None, :]).flatten(1)


def _factors(s):
    """scale of each row's adapter [M], 0 without one."""
    at = s["index"].long()
    return torch.where(at >= 0, s["scale"][at.clamp_min(0)], 0.0)


def _adapters(s):
    x, index, base = s["x"].float(), s["index"], s["base"].float()
    L = s["a"].shape[0]
    factor = _factors(s)
    if x.shape[0] <= L:  # few rows: their adapters, one copy a row
        at = index.long().clamp_min(0)
        h = (s["a"][at].float() * x[:, None, :]).sum(2) * (index >= 0)[:, None]
        y = base + (s["b"][at].float() * (h * factor[:, None])[:, :, None]).sum(1)
    else:  # many: every adapter, and what is not a row's own left out
        h, kept = _spread(x @ s["a"].float().flatten(0, 1).t(), index, L)
        y = base + (kept * factor[:, None]) @ s["b"].float().flatten(0, 1)
    return {"y": y.to(s["base"].dtype), "h": h}


def _adapter_grad(s):
    x, dy, index = s["x"].float(), s["dy"].float(), s["index"]
    a, b = s["a"].float().flatten(0, 1), s["b"].float().flatten(0, 1)
    L = s["a"].shape[0]
    factor = _factors(s)[:, None]
    dh = _spread(dy @ b.t(), index, L)[1] * factor
    dx = s["base"].float() + dh @ a
    db = _place(s["h"] * factor, index, L).t() @ dy
    return {"dx": dx.to(s["base"].dtype), "da": (dh.t() @ x).view(s["a"].shape), "db": db.view(s["b"].shape)}


def _member(seq, S):
    """Which sequence each row is of, as a matrix of zeros and ones [S, M]."""
    return (torch.arange(S, device=DEV)[:, None] == seq).float()


def _counts(index, E, seq, S):
    """Slots of each expert, int32 [S, E], and rows with any slot, [S], of each sequence."""
    slots = (index[:, :, None] == torch.arange(E, device=DEV)).sum(1)
    member = _member(seq, S)
    count = member @ slots.float()  # whole numbers below 2^24: exact
    return count.int(), (member @ (index >= 0).any(1).float()).int()


def _coef(count, rows):
    whole = count.sum(1, keepdim=True).double() * rows[:, None]
    return torch.where(whole > 0, count.shape[1] * count / whole, 0.0).float()


def _scores(l, score):
    """p and t of float logits, zeros at -inf."""
    ok = l > -math.inf
    if score == "softmax":
        e = torch.where(ok, torch.exp(l - l.amax(1, keepdim=True).clamp_min(torch.finfo(l.dtype).min)), 0)
        p = e
    else:
        p = e = torch.where(ok, 1 / (1 + torch.exp(-l)), 0)
    total = e.sum(1, keepdim=True)
    t = torch.where(total > 0, e / total, 0)
    return (t if score == "softmax" else p), t


def _balance(s, c):
    seq, S = _of_rows(c, s), c["S"]
    t = _scores(s["logits"].float(), c["score"])[1]
    count, rows = _counts(s["index"], c["E"], seq, S)
    coef = _coef(count, rows)
    t = torch.where((s["index"] >= 0).any(1, keepdim=True), t, 0)
    return {"loss": (coef * (_member(seq, S) @ t)).sum(1), "count": count, "coef": coef}


def _route_grad(s, c):
    seq, S = _of_rows(c, s), c["S"]
    p, t = _scores(s["logits"].float(), c["score"])
    some = s["index"] >= 0
    at = s["index"].long().clamp_min(0)
    chosen = torch.where(some, p.gather(1, at), 0)
    g = torch.where(some, s["dweight"] * c["factor"], 0)
    slope = p * (1 - p) if c["score"] == "sigmoid" else p  # of a sigmoid; a softmax takes off its mean below
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        inv = torch.where(total > 0, 1 / total, 0)
        g = (g - (g * chosen).sum(1, keepdim=True) * inv) * inv
    dp = torch.zeros_like(p).scatter_add_(1, at, torch.where(some, g, 0))
    dl = slope * dp
    if c["score"] == "softmax" and not c["renorm"]:
        dl -= p * (p * dp).sum(1, keepdim=True)
    counted = some.any(1) & (seq < S)
    to = seq.clamp_max(S - 1)
    q = torch.where(counted[:, None], s["coef"][to] * s["dloss"][to][:, None], 0)
    q = t * (q - (t * q).sum(1, keepdim=True))
    return (dl + (q * (1 - p) if c["score"] == "sigmoid" else q)).to(s["logits"].dtype)


def _own(s):
    import ternary_weight_linear_amd as tw

    c = s["case"]
    if c["op"] == "adapters":
        y, h = tw.bl_adapter_forward(s["x"], s["a"], s["b"], s["index"], scale=s["scale"], base=s["base"])
        return {"y": y, "h": h}
    if c["op"] == "adapter_grad":
        dx, da, db = tw.bl_adapter_backward(s["x"], s["a"], s["b"], s["index"], s["h"], s["dy"], scale=s["scale"], base=s["base"])
        return {"dx": dx, "da": da, "db": db}
    if c["op"] == "balance":
        loss, count, coef = tw.bl_route_balance(s["logits"], s["index"], score=c["score"], offsets=s["offsets"])
        return {"loss": loss, "count": count, "coef": coef}
    return tw.bl_route_backward(s["logits"], s["index"], dweight=s["dweight"], score=c["score"], renorm=c["renorm"], factor=c["factor"],
                                coef=s["coef"], dloss=s["dloss"], offsets=s["offsets"])


def run(state):
    if own:
        return _own(state)
    c = state["case"]
    if c["op"] == "adapters":
        return _adapters(state)
    if c["op"] == "adapter_grad":
        return _adapter_grad(state)
    return _balance(state, c) if c["op"] == "balance" else _route_grad(state, c)


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_adapters(s, c):
    x, base, scale = s["x"].double(), s["base"].double(), s["scale"].double()
    if c["op"] == "adapters":
        y, h = base.clone(), torch.zeros(c["M"], c["R"], dtype=torch.float64, device=DEV)
        for e in range(c["L"]):
            rows = (s["index"] == e).nonzero()[:, 0]
            if rows.numel():
                h[rows] = x[rows] @ s["a"][e].double().t()
                y[rows] += scale[e] * (h[rows] @ s["b"][e].double())
        return {"y": y, "h": h}
    dx, dy = base.clone(), s["dy"].double()
    da, db = torch.zeros(s["a"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["b"].shape, dtype=torch.float64, device=DEV)
    for e in range(c["L"]):
        rows = (s["index"] == e).nonzero()[:, 0]
        if rows.numel():
            dh = scale[e] * (dy[rows] @ s["b"][e].double().t())
            dx[rows] += dh @ s["a"][e].double()
            da[e] = dh.t() @ x[rows]
            db[e] = scale[e] * (s["h"][rows].double().t() @ dy[rows])
    return {"dx": dx, "da": da, "db": db}


def _exact_loss(s, c, logits):
    """Loss of each sequence, and the scores of all rows, by the definition."""
    E, bounds = c["E"], [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()
    gone = logits == -math.inf
    p = torch.sigmoid(logits).masked_fill(gone, 0) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(logits, 1))
    t = torch.nan_to_num(p / p.sum(1, keepdim=True))
    losses, coefs = [], []
    for at, end in zip(bounds[:-1], bounds[1:]):
        index = s["index"][at:end]
        rows = (index >= 0).any(1)
        count = torch.bincount(index[index >= 0].long(), minlength=E).double()
        whole = count.sum() * rows.sum()
        coefs.append(E * count / whole if whole > 0 else torch.zeros_like(count))
        losses.append((coefs[-1] * t[at:end][rows].sum(0)).sum())
    return torch.stack(losses), torch.stack(coefs), p


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] in ("adapters", "adapter_grad"):
        return _exact_adapters(s, c)
    if c["op"] == "balance":
        loss, coef, _ = _exact_loss(s, c, s["logits"].double())
        return {"loss": loss, "count": None, "coef": coef}
    logits = s["logits"].double()
    seen = logits > -math.inf
    # masked experts have no gradient: differentiate with respect to the others
    free = torch.where(seen, logits, 0).requires_grad_()
    loss, _, p = _exact_loss(s, c, torch.where(seen, free, -math.inf))
    some = s["index"] >= 0
    w = torch.where(some, p.gather(1, s["index"].long().clamp_min(0)), 0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, 1), 0)
    (c["factor"] * (w * s["dweight"]).sum() + (loss * s["dloss"].double()).sum()).backward()
    return torch.where(seen, torch.nan_to_num(free.grad), 0)
