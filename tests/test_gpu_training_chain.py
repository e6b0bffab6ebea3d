"""The operators of training beside frozen weights together, as a step of fine-tuning runs them: a
frozen 8-bit float layer with an adapter beside it, a frozen router with one, its choice and its
balance loss, forward and backward, against the formulas in 64 bits on what the frozen layers gave."""
import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

M, H, N, E, K, L, R = 96, 256, 384, 16, 4, 3, 8
u = 2.0 ** -24


def host(t):
    return t.double().cpu().numpy()


class Layer:
    """y = W x + s B^T (A x), W in e4m3 codes; its transpose, quantised once, takes gradients back."""

    def __init__(self, rows, cols, gen):
        w = torch.randn(rows, cols, generator=gen, device=DEV) * cols ** -0.5
        self.w, self.wt = tw.bl_fp8_quant_weight(w), tw.bl_fp8_quant_weight(w.t().contiguous())
        self.a = (torch.randn(L, R, cols, generator=gen, device=DEV) * cols ** -0.5).bfloat16()
        self.b = (torch.randn(L, R, rows, generator=gen, device=DEV) * 0.3).bfloat16()
        self.scale = torch.tensor([0.5, 2.0, 1.0], device=DEV)

    def forward(self, x, index):
        frozen = tw.bl_fp8_forward(x, *self.w)
        y, h = tw.bl_adapter_forward(x, self.a, self.b, index, scale=self.scale, base=frozen)
        return y, h, frozen

    def backward(self, x, index, h, dy, **kw):
        frozen = tw.bl_fp8_forward(dy, *self.wt)
        return *tw.bl_adapter_backward(x, self.a, self.b, index, h, dy, scale=self.scale, base=frozen, **kw), frozen


def step(layer, router, x, index, offsets, target, grads):
    y, h, _ = layer.forward(x, index)
    hidden = y.bfloat16()
    logits, hr, _ = router.forward(hidden, index)
    weight, chosen = tw.bl_route_experts(logits, K, score="sigmoid")
    loss, count, coef = tw.bl_route_balance(logits, chosen, score="sigmoid", offsets=offsets)
    dweight = weight - target                       # of half the squared distance
    dlogits = tw.bl_route_backward(logits, chosen, dweight, score="sigmoid", coef=coef, dloss=torch.full_like(loss, 0.01), offsets=offsets)
    da, db = grads["router"]
    dhidden, _, _, _ = router.backward(hidden, index, hr, dlogits, da=da, db=db)
    da, db = grads["layer"]
    dx, _, _, _ = layer.backward(x, index, h, dhidden, da=da, db=db)
    return y, logits, weight, chosen, loss, count, dlogits, dhidden, dx


def setup(seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    layer, router = Layer(N, H, gen), Layer(E, N, gen)
    x = torch.randn(M, H, generator=gen, device=DEV).bfloat16()
    index = torch.arange(M, device=DEV, dtype=torch.int32) // 30 - 1      # -1, 0, 1, 2 in runs
    offsets = torch.tensor([0, 30, 60, 90], dtype=torch.int32, device=DEV)   # the last rows are padding
    target = torch.rand(M, K, generator=gen, device=DEV)
    return layer, router, x, index, offsets, target


def zeros(layer, router):
    return {n: (torch.zeros(l.a.shape, device=DEV), torch.zeros(l.b.shape, device=DEV)) for n, l in (("layer", layer), ("router", router))}


def test_a_step_against_the_formulas():
    say("training step")
    layer, router, x, index, offsets, target = setup(0)
    grads = zeros(layer, router)
    y, logits, weight, chosen, loss, count, dlogits, dhidden, dx = step(layer, router, x, index, offsets, target, grads)
    ih, hidden = index.cpu().numpy(), y.bfloat16()

    def check(got, ref, mag, n, what):
        assert np.all(np.abs(host(got) - ref) <= n * u * mag + u * np.abs(ref) + 2.0 ** -140), what

    # each operator on what the one before it gave
    for l, xin, out in ((layer, x, y), (router, hidden, logits)):
        _, h, frozen = l.forward(xin, index)
        ref, href, mag, hmag = oa.forward(host(xin), host(l.a), host(l.b), ih, host(l.scale), host(frozen))
        check(h, href, hmag, xin.shape[1] / 4 + 64, "h")
        check(out, ref, mag, xin.shape[1] / 4 + R + 72, "y")
    lh, ch = host(logits), chosen.cpu().numpy()
    assert np.allclose(host(weight), oa.route_weights(lh, ch, "sigmoid", True, 1.0), rtol=2e-5, atol=0)
    rloss, rcount, rcoef = oa.balance(lh, ch, "sigmoid", offsets.tolist())
    assert np.array_equal(count.cpu().numpy(), rcount) and np.allclose(host(loss), rloss, rtol=2e-5)
    ref, mag = oa.route_backward(lh, ch, "sigmoid", True, 1.0, host(weight - target), rcoef, np.full(3, 0.01), offsets.tolist())
    check(dlogits, ref, mag, 200, "dlogits")
    for l, xin, dout, out, name in ((router, hidden, dlogits, dhidden, "router"), (layer, x, dhidden, dx, "layer")):
        _, h, _ = l.forward(xin, index)
        frozen = tw.bl_fp8_forward(dout, *l.wt)
        ref, mag = oa.backward(host(xin), host(l.a), host(l.b), ih, host(l.scale), host(h), host(dout), host(frozen))
        n = dout.shape[1] / 4 + M / 4 + R + 136
        check(out, ref["dx"], mag["dx"], n, "dx")
        check(grads[name][0], ref["da"], mag["da"], n, "da")
        check(grads[name][1], ref["db"], mag["db"], n, "db")


def test_gradients_of_the_adapters_against_differences():
    """The gradients of the router's adapter against differences of what the step minimises, the choice
    held by a step too small to change it: in 64 bits, with the frozen outputs as they came."""
    say("training differences")
    layer, router, x, index, offsets, target = setup(1)
    grads = zeros(layer, router)
    y, logits, weight, chosen, loss, count, *_ = step(layer, router, x, index, offsets, target, grads)
    hidden, ih, ch = host(y.bfloat16()), index.cpu().numpy(), chosen.cpu().numpy()
    frozen = host(tw.bl_fp8_forward(y.bfloat16(), *router.w))
    a, b, s, t = host(router.a), host(router.b), host(router.scale), host(target)

    def f(a, b):
        l = oa.forward(hidden, a, b, ih, s, frozen)[0]
        w = oa.route_weights(l, ch, "sigmoid", True, 1.0)
        return 0.5 * ((w - t) ** 2).sum() + 0.01 * oa.balance(l, ch, "sigmoid", offsets.tolist())[0].sum()

    g = np.random.default_rng(2)
    for at, grad, which in ((a, grads["router"][0], 0), (b, grads["router"][1], 1)):
        v = g.standard_normal(at.shape)
        d = 1e-5
        want = (f(a + d * v, b) - f(a - d * v, b)) / (2 * d) if which == 0 else (f(a, b + d * v) - f(a, b - d * v)) / (2 * d)
        assert abs((host(grad) * v).sum() - want) <= 1e-4 * np.abs(host(grad) * v).sum()


def test_the_step_from_a_graph_with_eager_work_between_replays():
    say("training graph")
    layer, router, x, index, offsets, target = setup(2)
    grads = zeros(layer, router)
    step(layer, router, x, index, offsets, target, grads)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for pair in grads.values():
            for t in pair:
                t.zero_()
        out = step(layer, router, x, index, offsets, target, grads)
    for turn in range(3):
        gen = torch.Generator(device=DEV).manual_seed(10 + turn)
        x.copy_(torch.randn(M, H, generator=gen, device=DEV).bfloat16())
        index.copy_(torch.randint(-1, L, (M,), generator=gen, device=DEV, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        eager = zeros(layer, router)
        want = step(layer, router, x, index, offsets, target, eager)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert all(torch.equal(a, b) for n in grads for a, b in zip(grads[n], eager[n]))
        torch.cuda.synchronize()
