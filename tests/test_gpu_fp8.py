"""GPU parity of the 8-bit floating point operators against the oracle: block quantisers (codes
and scales bit for bit), the block-scaled linear layer, routing to experts and the experts'
gated products."""
import numpy as np
import pytest
import torch

import oracle.fp8 as of
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
# Rounding of one result to its type (half a unit in the last place), and least step.
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
LEAST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -149}
# A block's sum from the matrix cores, relative to the sum of its magnitudes. fp16 operands: at
# most 128 roundings of fp32. e4m3 operands (16-bit results): terms keep 13 bits or more below
# the largest of a 32-term group, so a group errs by at most 32 2^-13 of its largest term; that
# largest term is what bounds it, 2^-8 of the magnitudes.
SUM = {"fp16": 2.0 ** -8, "bf16": 2.0 ** -8, "fp32": 2.0 ** -17}


def act(shape, dtype, seed, spread=1.0):
    """Values of the given type on the GPU, and the same in fp32 on the host."""
    g = np.random.default_rng(seed)
    v = g.standard_normal(shape) * np.exp(spread * g.standard_normal((shape[0], 1)))
    t = torch.from_numpy(v.astype(np.float32)).to(TYPES[dtype])
    return t.to(DEV), t.float().numpy()


def weight(N, K, seed):
    W = (np.random.default_rng(seed).standard_normal((N, K)) * K ** -0.5).astype(np.float32)
    codes, scales = of.quant_weight(W)
    return codes, scales


def f8(codes):
    return torch.from_numpy(np.ascontiguousarray(codes)).to(DEV).view(torch.float8_e4m3fn)


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def codes_of(t):
    return host(t.view(torch.uint8))


def close(y, ref, bound, dtype, what):
    y = y.float().cpu().numpy().astype(np.float64) if isinstance(y, torch.Tensor) else y
    err = np.abs(y - ref)
    tol = bound + UNIT[dtype] * (np.abs(ref) + bound) + LEAST[dtype]
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} out of tolerance, first at {i}: "
                             f"{y[i]!r} for {ref[i]!r}, allowed {tol[i]:.3g}")


# ------------------------------------------------------------------------------------------
# quantisers
# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 112), (5, 144), (16, 1024), (7, 8640), (129, 272)])
def test_quant_act(M, K, dtype):
    say("quant_act", M, K, dtype)
    x, v = act((M, K), dtype, 7 * M + K, spread=3.0)
    q, s = tw.bl_quant_act_fp8(x)
    c, sr, _ = of.quant_act(v)
    assert np.array_equal(codes_of(q), c)
    assert np.array_equal(host(s), sr)


def test_quant_act_of_every_fp16_value():
    """Each finite fp16 value in a row whose maximum is 65504, 1 or the value itself."""
    all16 = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16).view(np.float16)
    v = all16[np.isfinite(all16)].astype(np.float32)
    v = np.pad(v, (0, -v.size % 127)).reshape(-1, 127)
    for top in (65504.0, 1.0, 0.0):
        say("every fp16, top", top)
        rows = np.concatenate([np.full((v.shape[0], 1), top, np.float32), v if top > 1 else np.clip(v, -1, 1) if top else v], 1)
        x = torch.from_numpy(rows).half().to(DEV)
        q, s = tw.bl_quant_act_fp8(x)
        c, sr, _ = of.quant_act(x.float().cpu().numpy())
        assert np.array_equal(codes_of(q), c) and np.array_equal(host(s), sr)


def test_quant_act_rows_of_zeros_and_tiny_values():
    v = np.zeros((6, 256), np.float32)
    v[1, 3] = 1e-45                                # the least fp32 value
    v[2, :] = 2.0 ** -126
    v[3, 5] = -2.0 ** -100
    v[4, 130] = 3.4028235e38
    v[5, :] = -0.0
    q, s = tw.bl_quant_act_fp8(gpu(v))
    c, sr, _ = of.quant_act(v)
    assert np.array_equal(codes_of(q), c) and np.array_equal(host(s), sr)
    assert np.isfinite(host(s)).all()


def test_quant_act_of_nan_and_infinity():
    v = np.ones((3, 256), np.float32)
    v[0, 7] = np.nan
    v[1, 200] = -np.inf
    q, s = tw.bl_quant_act_fp8(gpu(v))
    val, sc = of.e4m3_values(codes_of(q)), host(s)
    assert np.isnan(val[0, :128]).all() and np.isnan(sc[0, 0])
    assert np.isnan(val[1, 200]) and np.isinf(sc[1, 1]) and (np.delete(val[1, 128:], 72) == 0).all()
    assert np.isfinite(val[0, 128:]).all() and np.isfinite(val[1, :128]).all() and np.isfinite(val[2]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,K", [(1, 16), (9, 272), (33, 1104)])
def test_quant_act_gated(M, K, dtype):
    """silu(gate) * up within a few roundings; codes equal except where the scaled value lies
    that near to a rounding boundary."""
    say("quant_act gated", M, K, dtype)
    x, v = act((M, 2 * K), dtype, 3 * M + K)
    q, s = tw.bl_quant_act_fp8(x, gated=True)
    h = of.silu_mul(v)
    c, sr, t = of.quant_act(h)
    rel = 8 * 2.0 ** -24                           # exp, sum, quotient, product, the scale's two steps
    assert np.all(np.abs(host(s) - sr) <= rel * sr)
    lo, hi = (of.e4m3_codes(np.abs(t) * (1 + d * 2 * rel)) for d in (-1, 1))
    got = codes_of(q)
    assert np.array_equal(got >= 128, c >= 128)
    assert np.all(((got & 127) == lo) | ((got & 127) == hi))


def test_quant_act_strided_rows():
    say("quant_act strided")
    x, v = act((9, 640), "bf16", 5)
    q, s = tw.bl_quant_act_fp8(x[:, 64:64 + 400])
    c, sr, _ = of.quant_act(v[:, 64:464])
    assert np.array_equal(codes_of(q), c) and np.array_equal(host(s), sr)


@pytest.mark.parametrize("N,K", [(1, 16), (128, 128), (129, 144), (200, 272), (384, 1040)])
def test_quant_weight(N, K):
    say("quant_weight", N, K)
    W = (np.random.default_rng(N + K).standard_normal((N, K)) * 0.02).astype(np.float32)
    W[0, :16] = 0
    codes, scales = tw.bl_fp8_quant_weight(gpu(W))
    c, s = of.quant_weight(W)
    assert np.array_equal(codes_of(codes), c) and np.array_equal(host(scales), s)


# ------------------------------------------------------------------------------------------
# linear layer
# ------------------------------------------------------------------------------------------
SHAPES = [(1, 1, 16), (1, 64, 128), (1, 100, 272), (2, 129, 1040), (3, 640, 8640), (5, 48, 400), (16, 256, 1024),
          (17, 130, 144), (33, 127, 640), (64, 128, 128), (65, 200, 272), (100, 257, 2064), (129, 384, 512),
          (200, 1000, 784), (257, 640, 1152), (300, 255, 4112), (513, 272, 256)]


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, out):
    dtype = ["fp16", "bf16", "fp32"][(M + N) % 3]
    say("fp8 linear", M, N, K, dtype, out)
    x, v = act((M, K), dtype, M + N + K)
    wc, ws = weight(N, K, N + K)
    y = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=TYPES[out])
    c, s, _ = of.quant_act(v)
    ref, mag = of.linear(c, s, wc, ws)
    assert y.dtype == TYPES[out] and tuple(y.shape) == (M, N)
    close(y, ref, (SUM[out] + (K // 128 + 4) * 2.0 ** -23) * mag, out, (M, N, K))
    two = tw.bl_fp8_linear(*tw.bl_quant_act_fp8(x), f8(wc), gpu(ws), out_dtype=TYPES[out])
    assert torch.equal(y, two)


@pytest.mark.parametrize("out", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1100, 8200, 272), (520, 8200, 400), (500, 6600, 656), (500, 3300, 1040), (300, 2500, 912),
                                   (40, 1000, 8208), (24, 28680, 400)])
def test_linear_wide(M, N, K, out):
    """Shapes of every tile that the product takes, odd rows, columns and blocks at their ends."""
    say("fp8 linear wide", M, N, K, out)
    x, v = act((M, K), "bf16", M)
    wc, ws = weight(N, K, K)
    y = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=TYPES[out])
    c, s, _ = of.quant_act(v)
    ref, mag = of.linear(c, s, wc, ws)
    close(y, ref, (SUM[out] + (K // 128 + 4) * 2.0 ** -23) * mag, out, (M, N, K))


@pytest.mark.parametrize("out", ["fp16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(300, 2100, 3104), (25, 300, 8208), (270, 4100, 8208), (1500, 1500, 272), (1601, 777, 8336),
                                   (412, 8645, 144), (728, 8239, 144), (69, 1702, 3760), (67, 5774, 4448), (130, 6406, 10016),
                                   (70, 8272, 11136), (421, 8246, 5584), (265, 11054, 6960), (2377, 7091, 1424), (195, 12384, 2704),
                                   (635, 14773, 2016), (13, 100, 2192), (9, 300, 4112), (16, 5000, 8208), (8, 16500, 2064)])
def test_linear_long_sums(M, N, K, out):
    """Every tile, whole, with K in parts, some of unequal lengths, and with the last tiles' in parts."""
    say("fp8 linear long sums", M, N, K, out)
    x, v = act((M, K), "fp16", M)
    wc, ws = weight(N, K, K)
    y = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=TYPES[out])
    c, s, _ = of.quant_act(v)
    ref, mag = of.linear(c, s, wc, ws)
    close(y, ref, (SUM[out] + (K // 128 + 4) * 2.0 ** -23) * mag, out, (M, N, K))
    assert torch.equal(y, tw.bl_fp8_linear(*tw.bl_quant_act_fp8(x), f8(wc), gpu(ws), out_dtype=TYPES[out]))


@pytest.mark.parametrize("M,N,K", [(1, 384, 1040), (16, 1000, 2064), (80, 640, 1152), (300, 513, 784)])
def test_linear_results_keep_the_precision_of_their_type(M, N, K):
    """Far below the worst-case bounds: fp32 results within fp32 roundings of the magnitudes of
    the sum (the roundings of K + K / 128 additions add up as their square root), 16-bit
    results within 1.01 units of rounding plus 2^-11 of the root of the summed squares (five
    times the 2^-16 per term of 128, over and over in the same direction)."""
    say("fp8 linear precision", M, N, K)
    x, v = act((M, K), "bf16", 1)
    wc, ws = weight(N, K, 2)
    c, s, _ = of.quant_act(v)
    ref, _ = of.linear(c, s, wc, ws)
    size = np.sqrt(np.square(of.act_values(c, s)) @ np.square(of.weight_values(wc, ws)).T)
    for out, extra in (("fp32", 2.0 ** -19), ("fp16", 2.0 ** -11), ("bf16", 2.0 ** -11)):
        y = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=TYPES[out]).float().cpu().numpy()
        assert np.all(np.abs(y - ref) <= 1.01 * UNIT[out] * np.abs(ref) + extra * size), out


def test_linear_is_exact_on_small_integers():
    """Integer inputs whose block maximum is 448 have scale 1 and are their own codes, so every
    sum is an integer below 2^24 and must come back exactly, whatever the order."""
    for M, N, K in ((1, 300, 1024), (20, 144, 528), (130, 257, 1024), (300, 640, 400)):
        say("fp8 linear exact", M, N, K)
        g = np.random.default_rng(M)
        x = g.integers(-8, 9, (M, K)).astype(np.float32)
        w = g.integers(-8, 9, (N, K)).astype(np.float32)
        x[:, ::128] = 448
        w[:, ::128] = 0
        w[::128, 1::128] = 448
        x[:, 1::128] = 0
        codes, scales = tw.bl_fp8_quant_weight(gpu(w))
        y = tw.bl_fp8_forward(gpu(x), codes, scales)
        assert np.array_equal(host(y), (x.astype(np.float64) @ w.T.astype(np.float64)).astype(np.float32))


def test_linear_places_every_input_and_output():
    """One-hot rows: y[m] is column 37 m + 5 (mod K) of w, so a misplaced input, block or output
    shows as a wrong value."""
    for M, N, K in ((3, 130, 400), (16, 272, 1040), (40, 500, 272), (256, 300, 784), (400, 129, 1152)):
        say("fp8 linear one-hot", M, N, K)
        wc, ws = weight(N, K, 9)
        x = np.zeros((M, K), np.float32)
        at = (37 * np.arange(M) + 5) % K
        x[np.arange(M), at] = 448.0
        y = host(tw.bl_fp8_forward(gpu(x), f8(wc), gpu(ws)))
        ref = 448.0 * of.weight_values(wc, ws)[:, at].T
        assert np.all(np.abs(y - ref) <= 2.0 ** -22 * np.abs(ref))


@pytest.mark.parametrize("M", [1, 16, 70, 300])
def test_linear_nan_and_infinity_stay_in_their_row_and_column(M):
    say("fp8 linear nan", M)
    N, K = 200, 400
    x, v = act((M, K), "fp32", 3)
    wc, ws = weight(N, K, 4)
    clean = host(tw.bl_fp8_forward(x, f8(wc), gpu(ws)))
    x[0, 399] = float("nan")
    if M > 1:
        x[M - 1, 17] = float("inf")
    wc = wc.copy()
    wc[131, 130] = 0x7F
    y = host(tw.bl_fp8_forward(x, f8(wc), gpu(ws)))
    bad = np.zeros((M, N), bool)
    bad[[0, M - 1]] = True
    bad[:, 131] = True
    assert np.isnan(y[bad]).all()
    assert np.array_equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("M", [4, 100, 300])
def test_linear_strided_rows_in_and_out(M):
    say("fp8 linear strided", M)
    N, K = 136, 272
    x, v = act((M, K + 64), "fp16", 6)
    wc, ws = weight(N, K, 7)
    for out in TYPES:
        room = torch.full((M, N + 5), 7.0, dtype=TYPES[out], device=DEV)
        y = tw.bl_fp8_forward(x[:, 32:32 + K], f8(wc), gpu(ws), out=room[:, 3:3 + N])
        plain = tw.bl_fp8_forward(x[:, 32:32 + K].contiguous(), f8(wc), gpu(ws), out_dtype=TYPES[out])
        assert torch.equal(y, plain)
        assert torch.all(room[:, :3] == 7) and torch.all(room[:, 3 + N:] == 7)


@pytest.mark.parametrize("M", [1, 16, 100, 300])
def test_linear_same_bits_on_every_run_and_stream(M):
    say("fp8 linear repeat", M)
    x, _ = act((M, 1040), "bf16", 8)
    wc, ws = weight(700, 1040, 9)
    w, s = f8(wc), gpu(ws)
    first = tw.bl_fp8_forward(x, w, s)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(tw.bl_fp8_forward(x, w, s))
    torch.cuda.synchronize()
    assert all(torch.equal(first, y) for y in got)


@pytest.mark.parametrize("M", [1, 24, 200])
def test_linear_replayed_from_a_graph(M):
    say("fp8 linear graph", M)
    x, _ = act((M, 528), "bf16", 10)
    wc, ws = weight(300, 528, 11)
    w, s = f8(wc), gpu(ws)
    y = torch.empty((M, 300), device=DEV)
    tw.bl_fp8_forward(x, w, s, out=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.bl_fp8_forward(x, w, s, out=y)
    for i in range(4):
        x.copy_(act((M, 528), "bf16", 20 + i)[0])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tw.bl_fp8_forward(x, w, s))


# ------------------------------------------------------------------------------------------
# routing
# ------------------------------------------------------------------------------------------
def grid_logits(M, E, seed):
    """Multiples of 1/4 in [-4, 4]: many ties, and different scores far apart."""
    return np.random.default_rng(seed).integers(-16, 17, (M, E)).astype(np.float32) / 4


ROUTES = [(1, 1, 1, 1, 1), (1, 256, 8, 8, 4), (7, 60, 4, 1, 1), (33, 64, 6, 8, 3), (5, 100, 64, 1, 1), (130, 512, 8, 16, 4),
          (3, 2048, 10, 64, 9), (9, 24, 3, 12, 5), (4, 65, 65 - 2, 1, 1), (6, 8, 2, 8, 2),
          (18, 120, 5, 8, 6), (5, 428, 4, 4, 2), (9, 264, 2, 8, 6), (3, 300, 16, 12, 4), (20, 406, 4, 2, 1), (2, 640, 9, 1, 1),
          (5, 51, 7, 3, 2), (4, 544, 3, 17, 6)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k,groups,kept", ROUTES)
def test_route(M, E, k, groups, kept, score):
    for dtype, biased, renorm in (("fp32", False, True), ("bf16", True, False), ("fp16", True, True)):
        say("route", M, E, k, groups, kept, score, dtype, biased)
        l = grid_logits(M, E, M + E)
        if biased and score == "softmax":
            l = l / 2                              # keeps different scores apart
        bias = (np.random.default_rng(E).integers(-2, 3, E) / 64).astype(np.float32) if biased else None
        ref_w, ref_i, gap = of.route(l, k, bias, score, groups, kept, renorm, 2.5)
        if gap < 1e-6:                             # undecided in fp32: drop the bias
            bias = None
            ref_w, ref_i, gap = of.route(l, k, bias, score, groups, kept, renorm, 2.5)
        assert gap > 1e-6
        w, i = tw.bl_route_experts(gpu(l).to(TYPES[dtype]), k, bias=None if bias is None else gpu(bias), score=score,
                                   groups=groups, kept_groups=kept, renorm=renorm, factor=2.5)
        assert np.array_equal(host(i), ref_i)
        # exp, its sum over E terms, the quotient, the sum over k and two more steps
        assert np.all(np.abs(host(w) - ref_w) <= (E ** 0.5 + k + 16) * 2.0 ** -23 * np.abs(ref_w) + 1e-37)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masked_rows_and_special_values(score):
    say("route special", score)
    inf, nan = np.inf, np.nan
    low = np.finfo(np.float32).min
    rows = np.array([[-inf] * 8, [nan] * 8, [-inf, 1, -inf, -inf, nan, -inf, 2, -inf], [low] * 8,
                     [low, low, 1, low, low, low, low, low], [inf, 0, inf, 0, 0, nan, 0, 0],
                     [0.0, -0.0, 0.0, -0.0, 0.0, -0.0, 0.0, -0.0], [-500, 0, 1, 2, 3, 4, 5, 500]], np.float32)
    for groups, kept, k in ((1, 1, 3), (4, 2, 3), (2, 2, 8), (4, 1, 2)):
        for renorm in (True, False):
            w, i = tw.bl_route_experts(gpu(rows), k, score=score, groups=groups, kept_groups=kept, renorm=renorm)
            ref_w, ref_i, _ = of.route(rows, k, None, score, groups, kept, renorm)
            assert np.array_equal(host(i), ref_i), (groups, kept, k)
            assert np.all(np.abs(host(w) - ref_w) <= 2.0 ** -19 * np.abs(ref_w) + 1e-37)
            assert (host(i)[:2] == -1).all() and (host(w)[:2] == 0).all()


def test_route_bias_that_is_not_finite():
    say("route bias")
    l = grid_logits(5, 16, 3)
    bias = np.zeros(16, np.float32)
    bias[2], bias[3], bias[5] = -np.inf, np.nan, np.inf
    w, i = tw.bl_route_experts(gpu(l), 14, bias=gpu(bias), score="sigmoid", renorm=False)
    i = host(i)
    assert (i[:, 0] == 5).all() and not np.isin(i, [2, 3]).any() and (i >= 0).all()
    assert np.isfinite(host(w)).all()


def test_route_strided_rows():
    say("route strided")
    l = grid_logits(9, 100, 4)
    w, i = tw.bl_route_experts(gpu(l)[:, 13:13 + 61], 5, score="sigmoid")
    ref_w, ref_i, _ = of.route(l[:, 13:74], 5, None, "sigmoid")
    assert np.array_equal(host(i), ref_i) and np.all(np.abs(host(w) - ref_w) <= 2.0 ** -19)


# ------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------
def expert_weights(E, H, I, seed):
    gu = [[weight(I, H, seed + 3 * e + i) for i in (0, 1)] for e in range(E)]
    d = [weight(H, I, seed + 3 * e + 2) for e in range(E)]
    wgu = np.stack([np.stack([c for c, _ in p]) for p in gu])
    sgu = np.stack([np.stack([s for _, s in p]) for p in gu])
    return wgu, sgu, np.stack([c for c, _ in d]), np.stack([s for _, s in d])


def choose(M, E, k, seed, away=0.0):
    g = np.random.default_rng(seed)
    index = np.stack([g.permutation(E)[:k] if k <= E else g.integers(0, E, k) for _ in range(M)]).astype(np.int32)
    index[g.random((M, k)) < away] = -1
    return index, g.random((M, k)).astype(np.float32)


EXPERTS = [(1, 4, 2, 16, 16), (1, 8, 8, 272, 144), (2, 3, 2, 512, 128), (7, 5, 3, 400, 272), (40, 6, 4, 256, 400),
           (150, 2, 1, 272, 144), (90, 3, 3, 144, 272), (500, 2, 1, 144, 272), (420, 1, 1, 400, 144)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("M,E,k,H,I", EXPERTS)
def test_experts(M, E, k, H, I, dtype):
    say("experts", M, E, k, H, I, dtype)
    x, v = act((M, H), dtype, M + H, spread=0.5)
    W = expert_weights(E, H, I, 100)
    index, wt = choose(M, E, k, 5, 0.2 if M > 2 else 0.0)
    y = tw.bl_fp8_experts(x, gpu(index), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3]))
    # fp32 sums of up to H or I terms; bf16 results take the e4m3 matrix instruction, whose
    # sums of 32 terms err by 2^-13 of the largest term
    rel = max(H, I) ** 0.5 * 2.0 ** -23 + (2.0 ** -12 if dtype == "bf16" else 2.0 ** -21)
    ref, bound = of.experts(v, index, wt, *W, rel)
    assert y.dtype == TYPES[dtype]
    close(y, ref, bound + 2.0 ** -20 * np.abs(ref).max(), dtype, (M, E, k, H, I))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,E,k,H,I", [(3201, 32, 2, 144, 528), (1601, 16, 1, 272, 528), (36, 9, 8, 400, 336),
                                       (3500, 32, 1, 272, 528)])
def test_experts_many_workgroups(M, E, k, H, I, dtype):
    """Enough workgroups for the large tiles of each type; many rows and few workgroups."""
    test_experts(M, E, k, H, I, dtype)


@pytest.mark.parametrize("M,E,k,times", [(700, 300, 4, 1), (100, 5, 8, 200), (60, 700, 2, 30)])
def test_experts_many_slots(M, E, k, times):
    """Enough slots that several workgroups sort them; repeated tokens get the same bits."""
    say("experts many slots", M * times, E, k)
    H = I = 16
    x, v = act((M, H), "fp32", M, spread=0.5)
    W = expert_weights(E, H, I, 200)
    index, wt = choose(M, E, k, 9, 0.1)
    many = [torch.cat([t] * times).contiguous() for t in (x, gpu(index), gpu(wt))]
    y = tw.bl_fp8_experts(*many, f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])).view(times, M, H)
    assert torch.equal(y, y[:1].expand(times, M, H))
    ref, bound = of.experts(v, index, wt, *W, H ** 0.5 * 2.0 ** -21)
    close(y[0], ref, bound + 2.0 ** -20 * np.abs(ref).max(), "fp32", (M, E, k))


def test_experts_slots_that_name_no_expert():
    """-1, out-of-range and repeated indices; a row without any expert gives zeros."""
    say("experts slots")
    M, E, k, H, I = 6, 3, 2, 144, 128
    x, v = act((M, H), "fp32", 1)
    W = expert_weights(E, H, I, 7)
    index = np.array([[-1, -1], [0, 0], [3, 1], [-7, 2], [2, -1], [1 << 30, -(1 << 31)]], np.int32)
    wt = np.ones((M, k), np.float32)
    y = host(tw.bl_fp8_experts(x, gpu(index), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])))
    ref, bound = of.experts(v, index, wt, *W, H ** 0.5 * 2.0 ** -22)
    close(y, ref, bound + 1e-6, "fp32", "slots")
    assert (y[[0, 5]] == 0).all() and not np.signbit(y[[0, 5]]).any()
    none = tw.bl_fp8_experts(x, gpu(np.full((M, k), -1, np.int32)), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3]))
    assert torch.all(none == 0)


@pytest.mark.parametrize("M", [3, 200])
def test_experts_nan_stays_in_its_token(M):
    say("experts nan", M)
    E, k, H, I = 4, 2, 272, 144
    x, v = act((M, H), "fp32", 2)
    W = expert_weights(E, H, I, 9)
    index, wt = choose(M, E, k, 3)
    args = gpu(index), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])
    clean = host(tw.bl_fp8_experts(x, *args))
    x[1, 100] = float("nan")
    y = host(tw.bl_fp8_experts(x, *args))
    assert np.isnan(y[1]).all()
    keep = np.arange(M) != 1
    assert np.array_equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 30, 300])
def test_experts_same_bits_on_every_run(M):
    say("experts repeat", M)
    E, k, H, I = 8, 4, 272, 272
    x, _ = act((M, H), "bf16", 4)
    W = expert_weights(E, H, I, 11)
    index, wt = choose(M, E, k, 6, 0.1)
    args = gpu(index), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])
    first = tw.bl_fp8_experts(x, *args)
    assert all(torch.equal(first, tw.bl_fp8_experts(x, *args)) for _ in range(4))
    # a token's result does not depend on the others: alone it takes another kernel, so equal
    # within the bounds of both
    one = tw.bl_fp8_experts(x[:1], gpu(index[:1]), gpu(wt[:1]), *args[2:])
    assert torch.allclose(one.float(), first[:1].float(), rtol=2.0 ** -6, atol=2.0 ** -6 * first[:1].float().abs().max().item())


def test_experts_strided_rows_and_other_output_types():
    say("experts strided")
    M, E, k, H, I = 20, 4, 2, 272, 144
    x, _ = act((M, H + 64), "bf16", 5)
    W = expert_weights(E, H, I, 13)
    index, wt = choose(M, E, k, 8)
    args = gpu(index), gpu(wt), f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])
    for out in TYPES:
        room = torch.full((M, H + 7), 3.0, dtype=TYPES[out], device=DEV)
        y = tw.bl_fp8_experts(x[:, 16:16 + H], *args, out=room[:, 2:2 + H])
        assert torch.equal(y, tw.bl_fp8_experts(x[:, 16:16 + H].contiguous(), *args, out_dtype=TYPES[out]))
        assert torch.all(room[:, :2] == 3) and torch.all(room[:, 2 + H:] == 3)


def test_route_and_experts_together():
    """Router logits to expert outputs, as a decode step runs them, from a graph."""
    say("route + experts graph")
    M, E, k, H, I = 5, 16, 4, 272, 144
    x, v = act((M, H), "bf16", 6)
    W = expert_weights(E, H, I, 15)
    args = f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])
    logits = gpu(grid_logits(M, E, 1))

    def step(out=None):
        wt, ix = tw.bl_route_experts(logits, k, score="sigmoid", groups=4, kept_groups=2)
        return tw.bl_fp8_experts(x, ix, wt, *args, out=out)

    y = step().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out=y)
    for i in range(4):
        logits.copy_(gpu(grid_logits(M, E, 30 + i)))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, step())


def test_example_runs_the_operators_together(capsys):
    """The example's layer, prompt and decode; quantising activations to 3 bits of mantissa twice
    leaves about 2 x 2^-4 / sqrt(3) x sqrt(2) = 0.1 of each product's size at most."""
    say("example")
    import examples.experts_decode as ex
    error = ex.main(["--hidden", "512", "--inner", "272", "--experts", "16", "--top", "4", "--groups", "4",
                     "--kept-groups", "2", "--prompt", "40", "--tokens", "3"])
    assert 0 < error < 0.1
    assert "us per token" in capsys.readouterr().out
