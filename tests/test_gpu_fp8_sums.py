"""Precision of the 8-bit floating point products' sums on the GPU, against the oracle's 64 bits,
at the sizes that reach each tile and on inputs where sums of fewer than 32 bits would show."""
import numpy as np
import pytest
import torch

import oracle.fp8 as of
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, host, say

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def act(shape, dtype, seed, spread=0.5):
    """Values of the given type on the GPU, and the same in fp32 on the host."""
    g = np.random.default_rng(seed)
    v = g.standard_normal(shape) * np.exp(spread * g.standard_normal((shape[0], 1)))
    t = torch.from_numpy(v.astype(np.float32)).to(TYPES[dtype])
    return t.to(DEV), t.float().numpy()


def weight(N, K, seed):
    return of.quant_weight((np.random.default_rng(seed).standard_normal((N, K)) * K ** -0.5).astype(np.float32))


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def f8(codes):
    return gpu(codes).view(torch.float8_e4m3fn)


def values(t):
    return t.float().cpu().numpy().astype(np.float64)


def rounded(ref, dtype):
    """The nearest value of the type, in fp64."""
    return torch.from_numpy(ref).to(TYPES[dtype]).double().numpy()


# ------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------
def expert_weights(E, H, I, seed):
    gu = [[weight(I, H, seed + 3 * e + i) for i in (0, 1)] for e in range(E)]
    d = [weight(H, I, seed + 3 * e + 2) for e in range(E)]
    return (np.stack([np.stack([c for c, _ in p]) for p in gu]), np.stack([np.stack([s for _, s in p]) for p in gu]),
            np.stack([c for c, _ in d]), np.stack([s for _, s in d]))


def choose(M, E, k, seed):
    g = np.random.default_rng(seed)
    return (np.stack([g.permutation(E)[:k] for _ in range(M)]).astype(np.int32), g.random((M, k)).astype(np.float32))


def operands(W):
    return f8(W[0]), gpu(W[1]), f8(W[2]), gpu(W[3])


def experts_exact(v, index, weight, wgu, sgu, wd, sd):
    """The experts' weighted sum in fp64, codes as the definition decides them."""
    y = np.zeros(v.shape)
    xc, xs, _ = of.quant_act(v)
    for e in np.unique(index):
        m, j = np.nonzero(index == e)
        h = of.silu_mul(np.concatenate([of.linear(xc[m], xs[:, m], wgu[e, i], sgu[e, i])[0] for i in (0, 1)], 1))
        hc, hs, _ = of.quant_act(h)
        np.add.at(y, m, weight[m, j, None].astype(np.float64) * of.linear(hc, hs, wd[e], sd[e])[0])
    return y


def rms(a):
    return np.sqrt(np.mean(np.square(a), 1))


def most_rows_err_by_rounding(y, ref, dtype, share):
    """A row whose codes of silu(gate) * up are the exact ones errs (root mean square) as rounding
    its results does, and by `share` of them beside it. fp32 sums err by about 2^-21 of their
    size, so a code, of a relative step of 1/16 to 1/8, is another one in 1e-5 of cases, a row of
    2000 of them in 2 %, and 15 % of the rows may be such; sums that err by 2^-16 make it 50 %."""
    got, most = rms(y - ref), rms(rounded(ref, dtype) - ref) + share * rms(ref)
    other = float(np.mean(got > most))
    assert other <= 0.15, f"{other:.0%} of the rows err by more than their results' rounding"


# From some 40 to some 1200 rows for each expert, few and many workgroups: each tile height.
TILES = [(90, 9, 4, 272, 528), (300, 6, 4, 272, 528), (1601, 16, 4, 272, 528), (3201, 32, 4, 144, 528),
         (1300, 4, 2, 400, 1040), (2400, 4, 2, 528, 1040)]


@pytest.mark.parametrize("dtype,out", [("bf16", "fp32"), ("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"),
                                       ("fp16", "bf16"), ("fp32", "fp32")])
@pytest.mark.parametrize("M,E,k,H,I", TILES)
def test_experts_sums_have_32_bits(M, E, k, H, I, dtype, out):
    """Whatever the types of inputs and results. Beside the codes, bf16 results may show the down
    product's 16-bit sums: 2e-5."""
    say("experts sums", M, E, k, H, I, dtype, out)
    x, v = act((M, H), dtype, M + H)
    W = expert_weights(E, H, I, 100)
    index, wt = choose(M, E, k, 5)
    y = values(tw.bl_fp8_experts(x, gpu(index), gpu(wt), *operands(W), out_dtype=TYPES[out]))
    some = np.random.default_rng(1).permutation(M)[:128]
    most_rows_err_by_rounding(y[some], experts_exact(v[some], index[some], wt[some], *W), out, 2.0 ** -14)


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,E,H,I", [(300, 4, 272, 528), (1200, 4, 528, 1040), (2000, 16, 1040, 272)])
def test_experts_outputs_that_nearly_cancel(M, E, H, I, out):
    """Two experts alike but for 2^-9 of the down matrix's scales, with weights 1 and -1: the
    result is 2^-9 of either output, so that those have to be summed as fp32."""
    say("experts cancel", M, E, H, I, out)
    x, v = act((M, H), "bf16", M)
    wgu, sgu, wd, sd = expert_weights(E, H, I, 50)
    wgu, sgu, wd = (np.repeat(a[: E // 2], 2, 0) for a in (wgu, sgu, wd))
    sd = np.repeat(sd[: E // 2], 2, 0)
    sd[1::2] *= np.float32(1 + 2.0 ** -9)
    first = 2 * np.random.default_rng(3).integers(0, E // 2, M)
    index = np.stack([first, first + 1], 1).astype(np.int32)
    wt = np.tile(np.array([1, -1], np.float32), (M, 1))
    y = values(tw.bl_fp8_experts(x, gpu(index), gpu(wt), f8(wgu), gpu(sgu), f8(wd), gpu(sd), out_dtype=TYPES[out]))
    some = np.random.default_rng(4).permutation(M)[:128]
    # the outputs' fp32 sums, within 2^-22, are 2^-13 of the result each
    most_rows_err_by_rounding(y[some], experts_exact(v[some], index[some], wt[some], wgu, sgu, wd, sd), out, 2.0 ** -11)


# ------------------------------------------------------------------------------------------
# one loud channel in every block
# ------------------------------------------------------------------------------------------
def half_unit(ref, dtype):
    """Half a unit in the last place of the type at ref."""
    bits, least = {"fp16": (10, -14), "bf16": (7, -126), "fp32": (23, -126)}[dtype]
    return np.exp2(np.maximum(np.frexp(ref)[1] - 1, least) - bits - 1)


# Streamed, and each tile of each instruction, whole and with K in parts.
WIDTHS = [(1, 300, 1040), (16, 1000, 2064), (24, 900, 4112), (40, 1000, 8208), (64, 128, 128), (129, 384, 528),
          (300, 2100, 3104), (270, 4100, 8208), (500, 3300, 1040), (500, 6600, 656), (520, 8200, 400), (1601, 777, 2192),
          (421, 8246, 1584)]


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,N,K", WIDTHS)
def test_linear_with_a_loud_channel(M, N, K, out):
    """Positive values, in each block one channel 448 times the others: the small products add up
    to a tenth of the large one, and sums that dropped their low bits would all err the same way.
    Every result within its own rounding and that of an fp32 sum: 128 roundings of a block's
    magnitudes and one for each block; bf16 results within 7 2^-13 of the magnitudes beside it."""
    say("fp8 linear loud", M, N, K, out)
    g = np.random.default_rng(M + N)
    v = np.abs(g.standard_normal((M, K))).astype(np.float32) + np.float32(0.1)
    v[:, 77::128] = 448 * (1 + np.arange(v[:, 77::128].shape[1]) % 3)
    x = gpu(v).to(torch.bfloat16)
    w, s = of.quant_weight(np.abs(g.standard_normal((N, K))).astype(np.float32) * np.float32(K ** -0.5))
    c, sx, _ = of.quant_act(values(x).astype(np.float32))
    ref, mag = of.linear(c, sx, w, s)
    y = values(tw.bl_fp8_forward(x, f8(w), gpu(s), out_dtype=TYPES[out]))
    tol = half_unit(ref, out) * (1 + 2.0 ** -10) + (2.0 ** -17 + (K // 128 + 4) * 2.0 ** -23) * mag
    if out == "bf16":
        tol += 7 * 2.0 ** -13 * mag
    worst = float((np.abs(y - ref) / tol).max())
    assert worst <= 1, f"{worst} times the allowed error"


@pytest.mark.parametrize("M,E,k,H,I", [(300, 6, 4, 272, 528), (1300, 4, 2, 400, 1040)])
def test_experts_fp16_results_with_a_loud_channel(M, E, k, H, I):
    """As above in the down product: everything positive, every eighth channel of silu(gate) * up a
    few hundred times the others."""
    say("experts loud", M, E, k, H, I)
    g = np.random.default_rng(M)
    x = gpu(np.abs(g.standard_normal((M, H))).astype(np.float32)).half()
    pos = lambda n, m: np.abs(g.standard_normal((n, m))).astype(np.float32) / np.float32(m)
    gu, d = [], []
    for e in range(E):
        up = pos(I, H)
        up[3::8] *= 300
        gu.append([of.quant_weight(pos(I, H)), of.quant_weight(up)])
        d.append(of.quant_weight(pos(H, I)))
    W = (np.stack([np.stack([c for c, _ in p]) for p in gu]), np.stack([np.stack([s for _, s in p]) for p in gu]),
         np.stack([c for c, _ in d]), np.stack([s for _, s in d]))
    index, wt = choose(M, E, k, 6)
    y = values(tw.bl_fp8_experts(x, gpu(index), gpu(wt), *operands(W)))
    some = g.permutation(M)[:128]
    ref = experts_exact(values(x)[some].astype(np.float32), index[some], wt[some], *W)
    most_rows_err_by_rounding(y[some], ref, "fp16", 2.0 ** -14)
    # roundings to fp16, up to 2^-11 either way, leave 2^-15 or less in the mean over a row's
    # columns (and codes that are others touch few rows); low bits dropped of positive sums stay
    shift = abs(float(np.median(np.mean(y[some] / ref - 1, 1))))
    assert shift <= 2.0 ** -15, f"results are off by {shift:.3g} on average"
