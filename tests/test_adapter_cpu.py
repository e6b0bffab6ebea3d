"""The oracle of the adapters and the router's training (gradients against differences), and the
refusals of their calls, without a GPU. The addresses passed here are fake; every call fails a
host check before anything is queued."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw

lib = tw._lib
OK, NULL, SHAPE, ALIGN, ALIAS, WS, HIP, ARG, CAPACITY = range(9)


# ------------------------------------------------------------------------------------------
# oracle
# ------------------------------------------------------------------------------------------
def difference(f, at, direction, step=1e-5):
    return (f(at + step * direction) - f(at - step * direction)) / (2 * step)


def test_adapter_gradients_are_those_of_the_forward_pass():
    g = np.random.default_rng(0)
    M, K, N, L, R = 7, 11, 5, 3, 2
    x, a, b, dy = g.normal(size=(M, K)), g.normal(size=(L, R, K)), g.normal(size=(L, R, N)), g.normal(size=(M, N))
    index, scale = np.array([2, 0, -1, 2, 3, 0, 2]), np.array([0.5, 2.0, 1.5])
    base = g.normal(size=(M, N))
    h = oa.forward(x, a, b, index, scale, base)[1]
    d, _ = oa.backward(x, a, b, index, scale, h, dy, np.zeros((M, K)))

    def f(x, a, b):
        return (oa.forward(x, a, b, index, scale, base)[0] * dy).sum()

    for name, at in (("dx", x), ("da", a), ("db", b)):
        v = g.normal(size=at.shape)
        fs = {"dx": lambda t: f(t, a, b), "da": lambda t: f(x, t, b), "db": lambda t: f(x, a, t)}[name]
        assert abs(difference(fs, at, v) - (d[name] * v).sum()) < 1e-7 * np.abs(d[name] * v).sum()
    assert not d["da"][1].any() and not d["dx"][[2, 4]].any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_is_that_of_weights_and_loss(score, renorm):
    g = np.random.default_rng(1)
    M, E, k = 9, 6, 3
    logits = g.normal(size=(M, E)) * 2
    logits[2, 4], logits[5] = -np.inf, -np.inf
    index = np.argsort(-logits, 1)[:, :k].astype(np.int32)
    index[5], index[7, 1], index[8] = -1, index[7, 0], E         # no expert, one twice, out of range
    offsets, factor = [1, 4, 4, 8], 1.5
    dweight, dloss = g.normal(size=(M, k)), g.normal(size=3)
    coef = oa.balance(logits, index, score, offsets)[2]
    d, mag = oa.route_backward(logits, index, score, renorm, factor, dweight, coef, dloss, offsets)

    def f(l):
        seq = oa.sequence_of_rows(offsets, M)
        on = (seq >= 0) & ((index >= 0) & (index < E)).any(1)
        loss = (np.where(on, dloss[np.maximum(seq, 0)], 0)[:, None] * coef[np.maximum(seq, 0)] * oa.scores(l, score)[1]).sum()
        return (oa.route_weights(l, index, score, renorm, factor) * dweight).sum() + loss

    v = np.where(np.isfinite(logits), g.normal(size=(M, E)), 0)
    assert abs(difference(f, np.where(np.isfinite(logits), logits, -np.inf), v) - (d * v).sum()) < 1e-7 * np.abs(d * v).sum()
    assert np.all(np.abs(d) <= mag + 1e-15) and not d[~np.isfinite(logits)].any()


def test_balance_loss_of_even_and_uneven_loads():
    E, M = 4, 8
    even = np.arange(M)[:, None] % E
    loss, count, coef = oa.balance(np.zeros((M, E)), even, "softmax")
    assert np.allclose(loss, 1) and np.array_equal(count, np.full((1, E), 2)) and np.allclose(coef, 1 / M)
    one = np.zeros((M, 1), int)
    logits = np.full((M, E), -30.0)
    logits[:, 0] = 30
    for score in ("softmax", "sigmoid"):
        assert np.allclose(oa.balance(logits, one, score)[0], E)     # all to one expert, and certain of it
    loss, count, _ = oa.balance(logits, one, "softmax", [0, 3, 3, 5])
    assert np.allclose(loss, [E, 0, E]) and count[:, 0].tolist() == [3, 0, 2]


# ------------------------------------------------------------------------------------------
# refusals of the C entry points
# ------------------------------------------------------------------------------------------
def P(v):
    return ctypes.c_void_p(v)


at = {n: 0x10000000 * (i + 1) for i, n in enumerate(
    ["x", "a", "b", "index", "scale", "base", "y", "h", "ws", "dy", "dx", "da", "db", "logits", "offsets", "loss", "count", "coef",
     "dweight", "dloss", "dlogits"])}


def forward(**kw):
    v = dict(at, dtype=1, ydtype=1, M=4, K=64, ldx=64, L=2, R=8, N=32, ldbase=32, ldy=32, wsb=1 << 24) | kw
    p = lambda n: P(v[n])
    return lib.bl_adapter_forward(p("x"), v["dtype"], v["M"], v["K"], v["ldx"], p("a"), p("b"), v["L"], v["R"], v["N"], p("index"), p("scale"),
                                  p("base"), v["ldbase"], p("y"), v["ydtype"], v["ldy"], p("h"), p("ws"), v["wsb"], None)


def backward(**kw):
    v = dict(at, dtype=1, dydtype=1, dxdtype=1, M=4, K=64, ldx=64, L=2, R=8, N=32, lddy=32, ldbase=64, lddx=64, add=0, wsb=1 << 24) | kw
    p = lambda n: P(v[n])
    return lib.bl_adapter_backward(p("x"), v["dtype"], v["M"], v["K"], v["ldx"], p("a"), p("b"), v["L"], v["R"], v["N"], p("index"), p("scale"),
                                   p("h"), p("dy"), v["dydtype"], v["lddy"], p("base"), v["ldbase"], p("dx"), v["dxdtype"], v["lddx"],
                                   p("da"), p("db"), v["add"], p("ws"), v["wsb"], None)


def balance(**kw):
    v = dict(at, dtype=2, M=4, E=8, ld=8, k=2, score=0, S=1, wsb=1 << 24) | kw
    p = lambda n: P(v[n])
    return lib.bl_route_balance(p("logits"), v["dtype"], v["M"], v["E"], v["ld"], p("index"), v["k"], v["score"], p("offsets"), v["S"], p("loss"),
                                p("count"), p("coef"), p("ws"), v["wsb"], None)


def route_backward(**kw):
    v = dict(at, dtype=2, ddtype=2, M=4, E=8, ld=8, k=2, score=0, S=1, ldd=8) | kw
    p = lambda n: P(v[n])
    return lib.bl_route_backward(p("logits"), v["dtype"], v["M"], v["E"], v["ld"], p("index"), v["k"], v["score"], p("dweight"), 1, 1.0, p("coef"),
                                 p("dloss"), p("offsets"), v["S"], p("dlogits"), v["ddtype"], v["ldd"], None)


@pytest.mark.parametrize("call", [forward, backward])
def test_adapter_checks(call):
    for name in ("x", "a", "b", "index", "h") + (("y",) if call is forward else ("dy", "da", "db")):
        assert call(**{name: None}) == NULL, name
    for kw in (dict(M=0), dict(M=(1 << 20) + 1), dict(K=0, ldx=1), dict(N=0), dict(R=0), dict(R=257), dict(L=0), dict(L=1025), dict(ldx=63),
               dict(ldbase=31)):
        assert call(**kw) == SHAPE, kw
    assert call(dtype=3) == ARG
    for name in ("ydtype",) if call is forward else ("dydtype", "dxdtype"):
        assert call(**{name: 0}) == ARG and call(**{name: 7}) == ARG         # neither x's type nor fp32
    many = {} if call is backward else dict(M=1 << 17, wsb=1 << 28)       # a forward pass of few rows needs no workspace
    assert call(**many | dict(wsb=16)) == WS and call(ws=None, **many) == WS
    for name, off in (("x", 1), ("a", 1), ("b", 1), ("index", 2), ("scale", 2), ("h", 2), ("base", 1)):
        assert call(**{name: at[name] + off}) == ALIGN, name
    assert call(ws=at["ws"] + 8, **many) == ALIGN
    out, ld = ("y", "ldy") if call is forward else ("dx", "lddx")
    for name in ("x", "a", "b", "index", "scale", "h"):
        assert call(**{out: at[name]}) == ALIAS, name
    assert call(**{out: at["ws"]}, **many) == ALIAS
    assert call(base=at[out] + 2) == ALIAS                                   # neither out itself nor apart from it
    assert call(base=at[out], ldbase=128, **{ld: 64}) == ALIAS


def test_adapter_backward_checks_of_its_own():
    assert backward(dx=None) == ARG                                          # a base without dx
    assert backward(lddy=31) == SHAPE and backward(lddx=63) == SHAPE
    assert backward(da=at["da"] + 2) == ALIGN and backward(db=at["db"] + 1) == ALIGN
    assert backward(da=at["db"]) == ALIAS and backward(db=at["dy"]) == ALIAS and backward(da=at["x"]) == ALIAS


def test_route_checks():
    for name in ("logits", "index", "loss", "count", "coef"):
        assert balance(**{name: None}) == NULL, name
    for kw in (dict(M=0), dict(M=(1 << 30) + 1), dict(E=0), dict(E=2049, ld=2049), dict(S=0), dict(S=(1 << 20) + 1), dict(ld=7),
               dict(M=1 << 30, k=2)):
        assert balance(**kw) == SHAPE, kw
    for kw in (dict(k=0), dict(k=65), dict(k=(1 << 32) + 1), dict(score=2), dict(dtype=3), dict(offsets=None, S=2)):
        assert balance(**kw) == ARG, kw
    assert balance(wsb=16) == WS and balance(ws=None) == WS
    for name, off in (("logits", 2), ("index", 1), ("offsets", 2), ("loss", 2), ("count", 2), ("coef", 2), ("ws", 4)):
        assert balance(**{name: at[name] + off}) == ALIGN, name
    assert balance(loss=at["logits"]) == ALIAS and balance(count=at["index"]) == ALIAS and balance(coef=at["count"]) == ALIAS
    assert balance(ws=at["logits"]) == ALIAS
    for kw in (dict(logits=None), dict(index=None), dict(dlogits=None), dict(dweight=None, coef=None), dict(dloss=None)):
        assert route_backward(**kw) == NULL, kw
    for kw in (dict(M=0), dict(E=2049, ld=2049, ldd=2049), dict(ld=7), dict(ldd=7)):
        assert route_backward(**kw) == SHAPE, kw
    for kw in (dict(k=0), dict(k=65), dict(score=-1), dict(dtype=3), dict(ddtype=3), dict(offsets=None, S=2)):
        assert route_backward(**kw) == ARG, kw
    for name, off in (("logits", 2), ("index", 1), ("dweight", 2), ("coef", 2), ("dloss", 1), ("offsets", 2), ("dlogits", 2)):
        assert route_backward(**{name: at[name] + off}) == ALIGN, name
    for name in ("logits", "index", "dweight", "coef", "dloss", "offsets"):
        assert route_backward(dlogits=at[name]) == ALIAS, name


def test_workspace_sizes():
    f = lib.bl_adapter_workspace_bytes
    assert f(0, 64, 64, 1, 1, 0) == 0 and f(1, 64, 64, 1, 257, 0) == 0 and f(1, 64, 64, 1025, 1, 1) == 0
    assert f(1, 64, 64, 1, 1, 0) == 0 and f(4096, 64, 64, 1, 1, 0) == 0      # few rows, each by itself
    assert 0 < f(1, 64, 64, 1, 1, 1) < f(4096, 64, 64, 1, 1, 1)
    assert 0 < f(70000, 64, 64, 1, 1, 0) < f(70000, 64, 64, 1, 1, 1)
    # sorted places of 32 rows for each adapter at most, padded to tiles, with a rank of 16 or more
    assert f(4096, 8192, 8192, 64, 16, 0) >= (4096 + 32 * 65) * 17 * 4
    for R in (1, 15, 16, 17, 64, 65, 256):
        for M in (1, 31, 8192, 8193, 1 << 20):
            assert f(M, 100, 300, 1024, R, 1) % 256 == 0
    g = lib.bl_route_balance_workspace_bytes
    assert g(0, 4, 1) == 0 and g(4, 2049, 1) == 0 and g(4, 4, 0) == 0
    assert 0 < g(1, 4, 1) < g(4096, 256, 1) < g(4096, 256, 100)


# ------------------------------------------------------------------------------------------
# refusals of the binding
# ------------------------------------------------------------------------------------------
x, a, b = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 32, dtype=torch.bfloat16)
index, h, dy = torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8), torch.zeros(4, 32, dtype=torch.bfloat16)


@pytest.mark.parametrize("args,kw,match", [
    ((x.double(), a, b, index), {}, "float16, bfloat16 or float32"),
    ((x, a.float(), b, index), {}, "a must be torch.bfloat16"),
    ((x, a, b.half(), index), {}, "b must be torch.bfloat16"),
    ((x, a, b, index.long()), {}, "index must be torch.int32"),
    ((x, a, b, index[:3]), {}, "index must be"),
    ((x, a[:1], b, index), {}, "a must be"),
    ((x, a, b.transpose(1, 2), index), {}, "b must be contiguous"),
    ((x, a, b[0], index), {}, "three dimensions"),
    ((x.t(), a, b, index), {}, "contiguous"),
    ((x, a, b, index), dict(scale=torch.zeros(3)), "scale must be"),
    ((x, a, b, index), dict(base=torch.zeros(4, 31)), "base must be"),
    ((x, a, b, index), dict(base=torch.zeros(4, 32), out_dtype=torch.bfloat16), "base must be torch.bfloat16"),
    ((x, a, b, index), dict(base=torch.zeros(4, 32), out=torch.zeros(4, 32, dtype=torch.bfloat16)), "base must be torch.bfloat16"),
    ((x, a, b, index), dict(out_dtype=torch.float16), "out must be torch.bfloat16 or torch.float32"),
    ((x, a, b, index), dict(out=torch.zeros(4, 32), out_dtype=torch.bfloat16), "out must be"),
    ((x, a, b, index), {}, "GPU"),
])
def test_adapter_forward_refusals(args, kw, match):
    with pytest.raises(ValueError, match=match):
        tw.bl_adapter_forward(*args, **kw)


@pytest.mark.parametrize("args,kw,match", [
    ((x, a, b, index, h.half(), dy), {}, "h must be torch.float32"),
    ((x, a, b, index, h[:, :7].contiguous(), dy), {}, "h must be"),
    ((x, a, b, index, h, dy.half()), {}, "dy must be torch.bfloat16 or torch.float32"),
    ((x, a, b, index, h, dy[:, :31]), {}, "dy must be"),
    ((x, a, b, index, h, dy), dict(da=torch.zeros(2, 8, 64)), "together"),
    ((x, a, b, index, h, dy), dict(da=torch.zeros(2, 8, 64), db=torch.zeros(2, 8, 64)), "db must be"),
    ((x, a, b, index, h, dy), dict(da=torch.zeros(2, 8, 64).half(), db=torch.zeros(2, 8, 32)), "da must be torch.float32"),
    ((x, a, b, index, h, dy), dict(need_dx=False, base=torch.zeros(4, 64)), "not asked for"),
    ((x, a, b, index, h, dy), dict(base=torch.zeros(4, 32)), "base must be"),
    ((x, a, b, index, h, dy), {}, "GPU"),
])
def test_adapter_backward_refusals(args, kw, match):
    with pytest.raises(ValueError, match=match):
        tw.bl_adapter_backward(*args, **kw)


logits, chosen, off = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)


@pytest.mark.parametrize("args,kw,match", [
    ((logits, chosen), dict(score="tanh"), "score"),
    ((logits, chosen.long()), {}, "index must be torch.int32"),
    ((logits, chosen[:3]), {}, "index must be"),
    ((logits, chosen), dict(offsets=off.long()), "offsets must be torch.int32"),
    ((logits, chosen), dict(offsets=off[:1]), "offsets must be"),
    ((logits.t(), chosen), {}, "contiguous"),
    ((logits, chosen), {}, "GPU"),
])
def test_route_balance_refusals(args, kw, match):
    with pytest.raises(ValueError, match=match):
        tw.bl_route_balance(*args, **kw)


@pytest.mark.parametrize("kw,match", [
    ({}, "must be given"),
    (dict(coef=torch.zeros(1, 8)), "together"),
    (dict(dloss=torch.zeros(1), dweight=torch.zeros(4, 2)), "together"),
    (dict(dweight=torch.zeros(4, 3)), "dweight must be"),
    (dict(dweight=torch.zeros(4, 2).double()), "dweight must be torch.float32"),
    (dict(coef=torch.zeros(2, 8), dloss=torch.zeros(1)), "coef must be"),
    (dict(coef=torch.zeros(1, 8), dloss=torch.zeros(2)), "dloss must be"),
    (dict(dweight=torch.zeros(4, 2), out_dtype=torch.float64), "float16, bfloat16 or float32"),
    (dict(dweight=torch.zeros(4, 2), out=torch.zeros(4, 8), out_dtype=torch.float16), "out must be"),
    (dict(dweight=torch.zeros(4, 2)), "GPU"),
])
def test_route_backward_refusals(kw, match):
    with pytest.raises(ValueError, match=match):
        tw.bl_route_backward(logits, chosen, **kw)
