"""The 8-bit floating point operators without a GPU: refusals of the C ABI (fake addresses,
every call below fails a host check) and of the binding, size queries, and the oracle's e4m3
arithmetic against torch's type."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.fp8 as of
import ternary_weight_linear_amd as tw

OK, NULL, SHAPE, ALIGN, ALIAS, WS, HIP, ARG = range(8)
A, B, C, D, E_, F, G, Y, W_ = (0x100000000 * i for i in range(1, 10))   # far apart
F16, BF16, F32 = 0, 1, 2
lib = tw._lib


def _p(v):
    return None if v is None else ctypes.c_void_p(v)


def call(name, defaults, **kw):
    a = {**defaults, **kw}
    fn = getattr(lib, name)
    return fn(*[_p(v) if t is ctypes.c_void_p else v for v, t in zip(a.values(), fn.argtypes)])


QUANT = dict(x=A, dtype=F16, M=4, K=256, ldx=256, gated=0, q=B, scales=C, stream=None)
LINEAR = dict(q=A, sx=B, M=4, K=256, w=C, sw=D, N=100, y=Y, ydtype=F32, ldy=100, ws=W_, wsb=1 << 20, stream=None)
FORWARD = dict(x=A, dtype=F16, M=4, K=256, ldx=256, w=C, sw=D, N=100, y=Y, ydtype=F32, ldy=100, ws=W_, wsb=1 << 20,
               stream=None)
ROUTE = dict(logits=A, dtype=F32, M=4, E=64, ld=64, bias=None, score=1, groups=8, kept=4, k=8, renorm=1, factor=1.0,
             weight=B, index=C, stream=None)
EXPERTS = dict(x=A, dtype=BF16, M=4, H=256, ldx=256, index=B, weight=B + 4096, k=2, wgu=C, sgu=D, wd=E_, sd=F, E=8, I=144,
               y=Y, ydtype=BF16, ldy=256, ws=W_, wsb=1 << 30, stream=None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(q=None), NULL), (dict(scales=None), NULL),
    (dict(M=0), SHAPE), (dict(K=0, ldx=0), SHAPE), (dict(K=24, ldx=24), SHAPE), (dict(M=(1 << 20) + 1), SHAPE),
    (dict(ldx=240), SHAPE), (dict(gated=1), SHAPE), (dict(dtype=3), ARG), (dict(dtype=-1), ARG),
    (dict(x=A + 8), ALIGN), (dict(ldx=260), ALIGN), (dict(q=B + 8), ALIGN), (dict(scales=C + 2), ALIGN),
    (dict(q=A + 1024), ALIAS), (dict(scales=B + 512), ALIAS), (dict(scales=A + 16), ALIAS)])
def test_quant_refusals(kw, want):
    assert call("bl_quant_act_fp8", QUANT, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), NULL), (dict(sx=None), NULL), (dict(w=None), NULL), (dict(sw=None), NULL), (dict(y=None), NULL),
    (dict(M=0), SHAPE), (dict(N=0), SHAPE), (dict(K=-16), SHAPE), (dict(K=120), SHAPE), (dict(ldy=99), SHAPE),
    (dict(ydtype=7), ARG), (dict(q=A + 4), ALIGN), (dict(w=C + 8), ALIGN), (dict(sx=B + 1), ALIGN), (dict(y=Y + 2), ALIGN),
    (dict(y=C + 16), ALIAS), (dict(y=A), ALIAS), (dict(y=D), ALIAS), (dict(ws=None), WS), (dict(wsb=64), WS),
    (dict(ws=W_ + 4), ALIGN), (dict(ws=B), ALIAS)])
def test_linear_refusals(kw, want):
    assert call("bl_fp8_linear", LINEAR, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(y=None), NULL), (dict(M=0), SHAPE), (dict(K=40, ldx=40), SHAPE), (dict(ldx=128), SHAPE),
    (dict(dtype=9), ARG), (dict(ydtype=9), ARG), (dict(x=A + 2), ALIGN), (dict(ws=None), WS), (dict(wsb=100), WS),
    (dict(ws=W_ + 4), ALIGN), (dict(y=A + 4), ALIAS), (dict(ws=A), ALIAS), (dict(ws=Y), ALIAS)])
def test_forward_refusals(kw, want):
    assert call("bl_fp8_forward", FORWARD, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(logits=None), NULL), (dict(weight=None), NULL), (dict(index=None), NULL), (dict(M=0), SHAPE), (dict(E=0), SHAPE),
    (dict(E=4096, ld=4096), SHAPE), (dict(ld=63), SHAPE), (dict(score=2), ARG), (dict(groups=0), ARG), (dict(groups=7), ARG),
    (dict(kept=9), ARG), (dict(kept=0), ARG), (dict(k=0), ARG), (dict(k=33), ARG), (dict(k=65, kept=8), ARG),
    (dict(dtype=4), ARG), (dict(index=C + 1), ALIGN), (dict(bias=D + 2), ALIGN), (dict(logits=A + 2), ALIGN),
    (dict(index=B + 64), ALIAS), (dict(weight=A + 64), ALIAS)])
def test_route_refusals(kw, want):
    assert call("bl_route_experts", ROUTE, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), NULL), (dict(index=None), NULL), (dict(weight=None), NULL), (dict(wgu=None), NULL), (dict(sd=None), NULL),
    (dict(M=0), SHAPE), (dict(k=0), SHAPE), (dict(k=65), SHAPE), (dict(E=0), SHAPE), (dict(E=4097), SHAPE),
    (dict(H=264, ldx=264), SHAPE), (dict(I=100), SHAPE), (dict(M=1 << 20, k=2), SHAPE), (dict(ldx=128), SHAPE),
    (dict(ldy=255), SHAPE), (dict(dtype=3), ARG), (dict(ydtype=3), ARG), (dict(wd=E_ + 4), ALIGN), (dict(index=B + 2), ALIGN),
    (dict(ws=None), WS), (dict(wsb=1000), WS), (dict(ws=W_ + 8), ALIGN), (dict(y=A), ALIAS), (dict(y=W_), ALIAS),
    (dict(ws=C), ALIAS)])
def test_experts_refusals(kw, want):
    assert call("bl_fp8_experts", EXPERTS, **kw) == want


def test_quant_weight_refusals():
    f = lib.bl_fp8_quant_weight
    assert f(_p(A), 4, 24, _p(B), _p(C), None) == SHAPE
    assert f(None, 4, 32, _p(B), _p(C), None) == NULL
    assert f(_p(A + 4), 4, 32, _p(B), _p(C), None) == ALIGN
    assert f(_p(A), 4, 32, _p(A + 64), _p(C), None) == ALIAS


def test_size_queries():
    assert lib.bl_fp8_workspace_bytes(0, 1, 128) == 0 and lib.bl_fp8_workspace_bytes(1, 1, 100) == 0
    assert lib.bl_fp8_workspace_bytes(1, 0, 128) == 0
    assert lib.bl_fp8_workspace_bytes(5, 64, 272) >= 5 * 272 + 5 * 3 * 4
    assert lib.bl_fp8_workspace_bytes(64, 1024, 8192) >= 64 * 8192 + 64 * 64 * 4 + 2 * 64 * 1024 * 4   # K in parts
    assert lib.bl_fp8_experts_workspace_bytes(1, 256, 0, 4, 128) == 0
    assert lib.bl_fp8_experts_workspace_bytes(1, 256, 2, 4, 120) == 0
    small, large = (lib.bl_fp8_experts_workspace_bytes(m, 256, 2, 4, 128) for m in (1, 64))
    assert 0 < small < large


def test_binding_refusals():
    x = torch.zeros(4, 256, dtype=torch.float16)
    w = torch.zeros(100, 256, dtype=torch.float8_e4m3fn)
    s = torch.zeros(1, 2)
    with pytest.raises(ValueError, match="GPU"):
        tw.bl_fp8_forward(x, w, s)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        tw.bl_quant_act_fp8(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        tw.bl_quant_act_fp8(x.t())
    with pytest.raises(ValueError, match="w must be torch.float8_e4m3fn"):
        tw.bl_fp8_forward(x, w.float(), s)
    with pytest.raises(ValueError, match="scales of w"):
        tw.bl_fp8_forward(x, w, s[:, :1].contiguous())
    with pytest.raises(ValueError, match="score"):
        tw.bl_route_experts(x.float(), 2, score="tanh")
    with pytest.raises(ValueError, match="index must be torch.int32"):
        tw.bl_fp8_experts(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2), w, s, w, s)


def test_oracle_codes_match_the_type():
    g = torch.Generator().manual_seed(0)
    t = (torch.randn(100000, generator=g) * torch.exp(4 * torch.randn(100000, generator=g))).clamp(-448, 448)
    assert np.array_equal(of.e4m3_codes(t.numpy()), t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(of.E4M3, every, equal_nan=True)
    mid = ((of._POS[1:] + of._POS[:-1]) / 2)          # ties go to the even code
    assert np.array_equal(of.e4m3_codes(mid), torch.from_numpy(mid.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_oracle_linear_on_exact_integers():
    g = np.random.default_rng(0)
    x, w = g.integers(-8, 9, (5, 272)).astype(np.float32), g.integers(-8, 9, (130, 272)).astype(np.float32)
    x[:, ::128], w[:, ::128], w[::128, 1::128], x[:, 1::128] = 448, 0, 448, 0
    xc, xs, _ = of.quant_act(x)
    y, _ = of.linear(xc, xs, *of.quant_weight(w))
    assert np.array_equal(y, x.astype(np.float64) @ w.T.astype(np.float64))


def test_oracle_experts_without_quantisation_loss():
    """One expert whose products are exact: y = weight * D(silu(G x) * U x) up to the last
    quantisation's step of 1/16."""
    H = I = 128
    x = np.zeros((1, H), np.float32)
    x[0, 0], x[0, 1] = 448, 224
    eye = np.eye(128, dtype=np.float32)
    q = [of.quant_weight(eye / 256)] * 2
    wgu, sgu = np.stack([c for c, _ in q])[None], np.stack([s for _, s in q])[None]
    wd, sd = (a[None] for a in of.quant_weight(eye))
    y, bound = of.experts(x, np.array([[0, -1]]), np.array([[2.0, 5.0]]), wgu, sgu, wd, sd, 1e-7)
    g = x[0].astype(np.float64) / 256
    want = 2 * g / (1 + np.exp(-g)) * g
    assert np.all(np.abs(y[0] - want) <= want / 16 + 1e-12) and np.all(bound >= 0)
