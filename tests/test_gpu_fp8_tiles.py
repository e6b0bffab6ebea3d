"""bf16 results of the 8-bit floating point linear layer, exactly, at each of its tiles: whole, with
K in parts, and with the last tiles' K in parts; ragged ends on every axis."""
import numpy as np
import pytest
import torch

import oracle.fp8 as of
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, say
from tests.test_gpu_fp8_sums import act, choose, expert_weights, f8, gpu, half_unit, operands, rounded, values, weight

pytestmark = pytest.mark.gpu

SHAPES = [(1, 300, 1040), (16, 1000, 2064), (25, 900, 3216),                                     # streamed
          (33, 64, 272), (35, 64, 3248), (33, 65, 144), (194, 8166, 144), (1777, 65, 3760),       # 64 x 64, 128 x 64
          (136, 11375, 144), (955, 3987, 144), (67, 4193, 5344), (2482, 1539, 5552),              # 128 x 128, eight waves
          (273, 11395, 144), (932, 8147, 144), (961, 1341, 8688),                                 # 128 x 128, four waves
          (540, 9699, 272), (907, 7979, 288), (132, 4303, 11280),                                 # 256 x 128
          (777, 9424, 144), (1976, 7984, 144), (389, 5416, 8656)]                                 # 256 x 256


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bf16_results_of_small_integers(M, N, K):
    """Inputs whose block maximum is 448 have scale 1 and are their own codes; products of integers
    up to 8 are within 13 bits of each other and their sums below 2^24, so the result is the exact
    sum, rounded once. The ragged last block counts like any other."""
    say("fp8 bf16 integers", M, N, K)
    g = np.random.default_rng(M)
    x, w = (g.integers(-8, 9, s).astype(np.float32) for s in ((M, K), (N, K)))
    x[:, ::128], w[:, ::128] = 448, 0
    w[::128, 1::128], x[:, 1::128] = 448, 0
    codes, scales = tw.bl_fp8_quant_weight(gpu(w))
    y = tw.bl_fp8_forward(gpu(x), codes, scales, out_dtype=torch.bfloat16)
    same = values(y) == rounded((x @ w.T).astype(np.float64), "bf16")   # fp32 sums of such integers are exact
    assert same.all(), f"{(~same).sum()} of {same.size} differ, first at {tuple(np.argwhere(~same)[0])}"


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_bf16_results_of_one_hot_rows(M, N, K):
    """y[m] is column 37 m + 5 (mod K) of w: one product, two scales and one rounding."""
    say("fp8 bf16 one-hot", M, N, K)
    wc, ws = weight(N, K, 9)
    x = np.zeros((M, K), np.float32)
    at = (37 * np.arange(M) + 5) % K
    x[np.arange(M), at] = 448.0
    y = values(tw.bl_fp8_forward(gpu(x), f8(wc), gpu(ws), out_dtype=torch.bfloat16))
    ref = 448.0 * of.weight_values(wc, ws)[:, at].T
    worst = float((np.abs(y - ref) / (half_unit(ref, "bf16") + 2.0 ** -22 * np.abs(ref) + 1e-38)).max())
    assert worst <= 1, f"{worst} times the allowed error"


SPECIAL = [(1, 200, 400), (16, 200, 400), (40, 130, 656), (70, 200, 400), (300, 200, 400), (777, 9424, 144), (132, 4303, 11280)]


@pytest.mark.parametrize("out", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", SPECIAL)
def test_nan_and_infinity_stay_in_their_row_and_column(M, N, K, out):
    say("fp8 nan", M, N, K, out)
    x, _ = act((M, K), "bf16", 3)
    wc, ws = weight(N, K, 4)
    clean = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=getattr(torch, {"bf16": "bfloat16", "fp16": "float16"}[out]))
    x[0, K - 1] = float("nan")
    if M > 1:
        x[M - 1, 17] = float("inf")
    wc = wc.copy()
    wc[121, 130] = 0x7F
    y = tw.bl_fp8_forward(x, f8(wc), gpu(ws), out_dtype=clean.dtype)
    bad = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    bad[[0, M - 1]] = True
    bad[:, 121] = True
    assert bool(torch.isnan(y[bad]).all())
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("M,N,K", [(35, 64, 3248), (540, 9699, 272), (389, 5416, 8656), (1976, 7984, 144)])
def test_bf16_same_bits_on_every_run_and_from_a_graph(M, N, K):
    say("fp8 bf16 repeat", M, N, K)
    x, _ = act((M, K), "bf16", 8)
    wc, ws = weight(N, K, 9)
    w, s = f8(wc), gpu(ws)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=DEV)
    tw.bl_fp8_forward(x, w, s, out=y)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got.append(tw.bl_fp8_forward(x, w, s, out_dtype=torch.bfloat16))
    torch.cuda.synchronize()
    assert all(torch.equal(y, t) for t in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.bl_fp8_forward(x, w, s, out=y)
    for i in range(3):
        x.copy_(act((M, K), "bf16", 20 + i)[0])
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, tw.bl_fp8_forward(x, w, s, out_dtype=torch.bfloat16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,E,k,H,I", [(3, 4, 2, 272, 144), (90, 9, 4, 272, 528), (300, 6, 4, 272, 528), (3201, 32, 4, 144, 528)])
def test_experts_nan_and_infinity_stay_in_their_token(M, E, k, H, I, dtype):
    """In an input, and in one expert's weights: its tokens and no others."""
    say("experts nan", M, E, k, H, I, dtype)
    x, _ = act((M, H), dtype, 2)
    W = expert_weights(E, H, I, 9)
    index, wt = choose(M, E, k, 3)
    call = lambda w: tw.bl_fp8_experts(x, gpu(index), gpu(wt), *operands(w))
    clean = call(W)
    assert bool(torch.isfinite(clean).all())
    x[1, 100], x[M - 1, 5] = float("nan"), float("-inf")
    wd = W[2].copy()
    wd[0, 7, 130] = 0x7F                            # expert 0: channel 7 of its tokens
    y = call((W[0], W[1], wd, W[3]))
    bad = torch.zeros((M, H), dtype=torch.bool, device=DEV)
    bad[[1, M - 1]] = True
    bad[gpu((index == 0).any(1)), 7] = True
    assert bool(torch.isnan(y[bad]).all())
    assert torch.equal(y[~bad], clean[~bad])
