"""An adapter beside each of the low-bit layers, and the gradient that passes such a frozen layer: the
layer of its transposed codes, which is what the adapter's dx is added onto."""
import numpy as np
import pytest

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import say
from tests.test_gpu_adapter import close, gpu, host, u

pytestmark = pytest.mark.gpu

K, N, L, R = 256, 384, 3, 8


def ternary(g):
    codes, beta = g.integers(-1, 2, (N, K)).astype(np.int8), np.float32(0.03)
    packed = [gpu(c) for c in (codes, codes.T)]
    fw, bw = (tw.bl_pack_ternary(c) for c in packed)
    b = gpu(np.array([beta]))

    def backward(dy):
        # of dy in int8, each value off by half a step, max|dy| / 254
        dyh = host(dy)
        slack = beta * np.abs(dyh).max(1, keepdims=True) / 254 * np.abs(codes).sum(0)
        return tw.bl_bitlinear_forward(dy, bw, b, K), beta * (dyh @ codes), 1.001 * slack
    return lambda x: tw.bl_bitlinear_forward(x, fw, b, N), backward


def onebit(g):
    s = np.where(g.random((N, K)) < 0.5, -1.0, 1.0)
    cols, rows = (g.uniform(0.5, 1.5, n).astype(np.float16) for n in (K, N))
    fw, bw = (tw.bl_pack_sign(gpu(np.ascontiguousarray(m).astype(np.float32))) for m in (s, s.T))

    def backward(dy):
        dyh, c, r = host(dy), cols.astype(np.float64), rows.astype(np.float64)
        return tw.bl_onebit_linear(dy, gpu(rows), bw, gpu(cols)), c * ((r * dyh) @ s), 1e-3 * c * (np.abs(r * dyh).sum(1, keepdims=True))
    return lambda x: tw.bl_onebit_linear(x, gpu(cols), fw, gpu(rows)), backward


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("layer", [ternary, onebit])
def test_an_adapter_beside_a_low_bit_layer(layer, M):
    say("adapter beside", layer.__name__, M)
    g = np.random.default_rng(M)
    forward, backward = layer(g)
    half = lambda *shape, size=1.0: gpu((g.standard_normal(shape) * size).astype(np.float16))
    x, a, b, dy = half(M, K), half(L, R, K, size=K ** -0.5), half(L, R, N, size=0.3), half(M, N)
    index, scale = g.integers(-1, L, M).astype(np.int32), np.array([0.5, 2.0, 1.0], np.float32)
    y = forward(x)
    base = host(y)
    y, h = tw.bl_adapter_forward(x, a, b, gpu(index), scale=gpu(scale), base=y, out=y)
    ref, href, mag, hmag = oa.forward(host(x), host(a), host(b), index, scale, base)
    close(h, href, (K / 4 + 64) * u * hmag, "fp32", "h")
    close(y, ref, (K / 4 + R + 72) * u * mag + u * np.abs(ref), "fp32", "y")
    dx, want, slack = backward(dy)
    through = host(dx)
    assert np.all(np.abs(through - want) <= slack + 1e-5 * np.abs(want))
    dx, da, db = tw.bl_adapter_backward(x, a, b, gpu(index), h, dy, scale=gpu(scale), base=dx, out=dx)
    ref, mag = oa.backward(host(x), host(a), host(b), index, scale, host(h), host(dy), through)
    close(dx, ref["dx"], (N / 4 + R + 72) * u * mag["dx"] + u * np.abs(ref["dx"]), "fp32", "dx")
    close(da, ref["da"], (N / 4 + M / 4 + 136) * u * mag["da"] + u * np.abs(ref["da"]), "fp32", "da")
    close(db, ref["db"], (M / 4 + 72) * u * mag["db"] + u * np.abs(ref["db"]), "fp32", "db")
