"""GPU parity of the balance loss and the router's gradient against the oracle in 64 bits.

Bounds. u = 2^-24 is half a unit of fp32. A score t takes an exponential of a rounded difference
(an error of u |l - max| in its argument, two units of its own), a division, and a sum of E positive terms in
chains of at most E / 16 + 4 roundings; sigmoids take two of each. So t is within
(2 |l - max| + E / 8 + 40) u of itself, and what is made of it by products and sums of few terms within
that of the sum of its magnitudes, a sum over E again included."""
import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
LEAST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -126}     # results below 2^-126 may be 0
u = 2.0 ** -24


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.double().cpu().numpy()


def make(M, E, k, dtype, seed, masked=0.0, size=1.5):
    """(logits, the same in 64 bits, index int32 on the host)."""
    g = np.random.default_rng(seed)
    l = g.standard_normal((M, E)) * size
    l[g.random((M, E)) < masked] = -np.inf
    t = torch.from_numpy(l.astype(np.float32)).to(TYPES[dtype])
    lh = t.double().numpy()
    index = np.argsort(-lh, 1, kind="stable")[:, :k].astype(np.int32)
    index[np.take_along_axis(lh, index, 1) == -np.inf] = -1
    return t.to(DEV), lh, index


def rounding(lh, E):
    """The relative bound of each row's scores."""
    l = np.where(np.isfinite(lh), lh, np.nan)
    with np.errstate(all="ignore"):
        span = np.nan_to_num(np.nanmax(np.where(np.isnan(l).all(1, keepdims=True), 0, l), 1) - np.nanmin(np.where(np.isnan(l).all(1, keepdims=True), 0, l), 1))
    return ((2 * span + E / 8 + 40) * u)[:, None]


def check_balance(got, lh, index, score, offsets=None):
    loss, count, coef = got
    rloss, rcount, rcoef = oa.balance(lh, index, score, offsets)
    assert loss.dtype == coef.dtype == torch.float32 and count.dtype == torch.int32
    assert np.array_equal(count.cpu().numpy(), rcount)
    assert np.all(np.abs(host(coef) - rcoef) <= 2 * u * rcoef)
    M, E = lh.shape
    rows = M // 512 // 16 + 40                     # additions of a chunk's sums
    assert np.all(np.abs(host(loss) - rloss) <= (rounding(lh, E).max() + rows * u) * rloss + 1e-37), (host(loss), rloss)


def check_gradient(got, lh, index, score, renorm, factor, out, **kw):
    ref, mag = oa.route_backward(lh, index, score, renorm, factor, **kw)
    assert got.dtype == TYPES[out]
    bound = 2 * rounding(lh, lh.shape[1]) * mag
    tol = bound + UNIT[out] * (np.abs(ref) + bound) + LEAST[out]
    err = np.abs(host(got) - ref)
    bad = ~(err <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{bad.sum()} of {bad.size} out of tolerance, first at {i}: {host(got)[i]!r} for {ref[i]!r}, allowed {tol[i]:.3g}")


SHAPES = [(1, 1, 1), (1, 256, 8), (3, 2, 2), (40, 60, 4), (33, 64, 1), (17, 100, 16), (100, 128, 17), (65, 250, 6), (50, 257, 8), (9, 300, 64),
          (30, 512, 3), (21, 513, 9), (10, 1000, 40), (7, 2047, 5), (5, 2048, 64), (1500, 48, 2), (700, 8, 8)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,k", SHAPES)
def test_balance_and_gradient(M, E, k, score):
    for i, dtype in enumerate(TYPES):
        masked = (0.0, 0.3, 0.9)[(M + i) % 3]
        say("route grad", M, E, k, score, dtype, masked)
        logits, lh, index = make(M, E, k, dtype, M + E + i, masked)
        got = tw.bl_route_balance(logits, gpu(index), score=score)
        check_balance(got, lh, index, score)
        dweight = np.random.default_rng(1).standard_normal((M, k)).astype(np.float32)
        dloss = np.array([1.7], np.float32)
        for renorm in (False, True):
            out = list(TYPES)[(i + renorm) % 3]
            kw = dict(score=score, renorm=renorm, factor=2.5, out_dtype=TYPES[out])
            d = tw.bl_route_backward(logits, gpu(index), gpu(dweight), coef=got[2], dloss=gpu(dloss), **kw)
            check_gradient(d, lh, index, score, renorm, 2.5, out, dweight=dweight, coef=host(got[2]), dloss=dloss)
        d = tw.bl_route_backward(logits, gpu(index), gpu(dweight), score=score, renorm=bool(M % 2))
        check_gradient(d, lh, index, score, bool(M % 2), 1.0, dtype, dweight=dweight)
        d = tw.bl_route_backward(logits, gpu(index), coef=got[2], dloss=gpu(dloss), score=score, out_dtype=torch.float32)
        check_gradient(d, lh, index, score, True, 1.0, "fp32", coef=host(got[2]), dloss=dloss)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,E,offsets", [
    (64, 60, [0, 64]), (64, 60, [0, 1, 1, 1, 17, 64]), (100, 256, [5, 20, 90]), (300, 16, list(range(0, 301, 3))), (200, 600, [0, 0, 0, 200]),
    (50, 24, [50, 50]), (50, 24, [0, 60, 70]), (50, 24, [-9, -3, 20, 50, 999]), (3000, 30, [0, 7, 1500, 1501, 2999, 3000]), (1, 4, [0, 0, 1, 1]),
    (9000, 12, list(range(0, 9001, 90)))])
def test_packed_sequences(M, E, offsets, score):
    """Empty sequences, rows before the first and behind the last, offsets past the rows, more
    sequences than chunks of rows."""
    say("route sequences", M, E, len(offsets) - 1, score)
    logits, lh, index = make(M, E, 3, "fp32", M)
    index[::5] = -1                                # rows without an expert count nowhere
    off = np.array(offsets, np.int32)
    got = tw.bl_route_balance(logits, gpu(index), score=score, offsets=gpu(off))
    check_balance(got, lh, index, score, offsets)
    S = len(offsets) - 1
    dloss = np.random.default_rng(2).standard_normal(S).astype(np.float32)
    dweight = np.random.default_rng(3).standard_normal((M, 3)).astype(np.float32)
    d = tw.bl_route_backward(logits, gpu(index), gpu(dweight), score=score, coef=got[2], dloss=gpu(dloss), offsets=gpu(off))
    check_gradient(d, lh, index, score, True, 1.0, "fp32", dweight=dweight, coef=host(got[2]), dloss=dloss, offsets=offsets)
    none = oa.sequence_of_rows(offsets, M) < 0
    d = tw.bl_route_backward(logits, gpu(index), score=score, coef=got[2], dloss=gpu(dloss), offsets=gpu(off))
    assert not host(d)[none].any() and not host(d)[::5].any()


def test_falling_offsets_stay_inside_the_buffers():
    """Offsets that fall are outside the contract: any numbers may come back, but no other memory is reached."""
    say("route falling offsets")
    M, E = 500, 40
    logits, lh, index = make(M, E, 2, "fp32", 4)
    off = gpu(np.array([400, 100, 450, -5, 2 ** 31 - 1, 30, 500], np.int32))
    loss, count, coef = tw.bl_route_balance(logits, gpu(index), offsets=off)
    tw.bl_route_backward(logits, gpu(index), coef=coef, dloss=loss, offsets=off)
    torch.cuda.synchronize()
    got = tw.bl_route_balance(logits, gpu(index))
    check_balance(got, lh, index, "softmax")


@pytest.mark.parametrize("E", [6, 64, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_odd_logits(E, score):
    """NaN and -inf are left out, +inf counts as the largest finite value; far values keep their
    scores; a row without any gives zeros."""
    say("route odd logits", E, score)
    M = 12
    _, lh, index = make(M, E, 3, "fp32", 5)
    lh[0, 1], lh[1, 2], lh[2], lh[3] = np.nan, np.inf, -np.inf, np.nan
    lh[4] -= 200                                   # every sigmoid is below fp32's least value
    lh[5] += 300
    lh[6] = -3e38
    lh[7, 0] = 3e38
    lh[8] = 0
    index[9] = [2, 2, 4]                           # the same expert twice
    index[10] = [E, -7, 5]
    index[11] = [1, 1, 1]
    t = torch.from_numpy(lh.astype(np.float32)).to(DEV)
    lh = t.double().cpu().numpy()
    got = tw.bl_route_balance(t, gpu(index), score=score)
    check_balance(got, lh[:, :], index, score)
    for m in range(M):                             # each row by itself, where the others' sums hide nothing
        check_balance(tw.bl_route_balance(t[m:m + 1], gpu(index[m:m + 1]), score=score), lh[m:m + 1], index[m:m + 1], score)
    dweight = np.random.default_rng(6).standard_normal((M, 3)).astype(np.float32)
    for renorm in (True, False):
        rows = [m for m in range(M) if not (m == 4 and score == "sigmoid" and renorm)]   # the weights themselves are 0 there
        d = tw.bl_route_backward(t, gpu(index), gpu(dweight), score=score, renorm=renorm, coef=got[2], dloss=gpu(np.ones(1, np.float32)))
        ref = dict(dweight=dweight, coef=host(got[2]), dloss=np.ones(1))
        assert torch.isfinite(d).all()
        full, mag = oa.route_backward(lh, index, score, renorm, 1.0, **ref)
        bound = 2 * rounding(lh, E) * mag
        err = np.abs(host(d) - full)
        assert np.all((err <= bound + u * np.abs(full) + LEAST["fp32"])[rows])


def test_strided_rows():
    say("route strided")
    for shift, E in ((4, 60), (3, 60), (1, 33)):
        logits, lh, index = make(70, E, 4, "bf16", 7)
        room = torch.zeros((70, E + 8), dtype=torch.bfloat16, device=DEV)
        room[:, shift:shift + E] = logits
        view = room[:, shift:shift + E]
        got = tw.bl_route_balance(view, gpu(index))
        check_balance(got, lh, index, "softmax")
        dweight = np.random.default_rng(8).standard_normal((70, 4)).astype(np.float32)
        for out in TYPES:
            oroom = torch.full((70, E + 8), 7.0, dtype=TYPES[out], device=DEV)
            d = tw.bl_route_backward(view, gpu(index), gpu(dweight), coef=got[2], dloss=torch.ones(1, device=DEV), out=oroom[:, shift:shift + E])
            check_gradient(d, lh, index, "softmax", True, 1.0, out, dweight=dweight, coef=host(got[2]), dloss=np.ones(1))
            assert torch.all(oroom[:, :shift] == 7) and torch.all(oroom[:, shift + E:] == 7)


def test_same_bits_on_every_run_and_stream_and_from_a_graph():
    say("route repeat")
    M, E, k = 5000, 96, 6
    logits, lh, index = make(M, E, k, "bf16", 9)
    index[7] = [3, 3, 3, 5, 5, 1]
    idx, dw = gpu(index), gpu(np.random.default_rng(10).standard_normal((M, k)).astype(np.float32))
    off = gpu(np.array([0, 1000, 1003, 4800], np.int32))
    dl = gpu(np.array([0.5, 1.0, -2.0], np.float32))

    def step():
        got = tw.bl_route_balance(logits, idx, score="sigmoid", offsets=off)
        return (*got, tw.bl_route_backward(logits, idx, dw, score="sigmoid", coef=got[2], dloss=dl, offsets=off))

    first = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(4):
        with torch.cuda.stream(streams[i % 2]):
            got.append(step())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(first, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(3):
        logits.copy_(make(M, E, k, "bf16", 20 + turn)[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, step()))
        torch.cuda.synchronize()


def test_the_choice_of_bl_route_experts_and_its_gradient_by_differences():
    """Routing, its loss, and the directional derivative of both along a random direction, the
    choice held fixed: in 64 bits from the oracle's forward pass."""
    say("route chain")
    M, E, k = 64, 32, 4
    logits, lh, _ = make(M, E, k, "fp32", 11)
    for score in ("softmax", "sigmoid"):
        weight, index = tw.bl_route_experts(logits, k, score=score, groups=4, kept_groups=2, factor=1.5)
        ih = index.cpu().numpy()
        assert np.allclose(host(weight), oa.route_weights(lh, ih, score, True, 1.5), rtol=1e-5)
        loss, count, coef = tw.bl_route_balance(logits, index, score=score)
        g = np.random.default_rng(12)
        dweight, v = g.standard_normal((M, k)).astype(np.float32), g.standard_normal((M, E))
        d = tw.bl_route_backward(logits, index, gpu(dweight), score=score, factor=1.5, coef=coef, dloss=torch.ones_like(loss))

        def f(l):
            return (oa.route_weights(l, ih, score, True, 1.5) * dweight).sum() + oa.balance(l, ih, score)[0].sum()

        want = (f(lh + 1e-5 * v) - f(lh - 1e-5 * v)) / 2e-5
        assert abs((host(d) * v).sum() - want) <= 1e-5 * np.abs(host(d) * v).sum()


def test_more_rows_than_a_grid_has_work_items_along_x():
    """2^28 rows of 16 lanes each are 2^32 work-items; the last rows and all counts."""
    say("route many rows")
    M, E = (1 << 28) + 5, 2
    logits = torch.zeros((M, E), dtype=torch.bfloat16, device=DEV)
    index = torch.zeros((M, 1), dtype=torch.int32, device=DEV)
    index[1::4] = 1
    index[3::4] = -1
    tail, lh, _ = make(37, E, 1, "bf16", 13)
    logits[-37:] = tail
    dweight = torch.ones((M, 1), device=DEV)
    loss, count, coef = tw.bl_route_balance(logits, index)
    n = [(index == e).sum().item() for e in range(E)]
    assert count[0].tolist() == n
    # even scores but for the last rows: the loss is E (n_0 + n_1) / (2 C) = 1 to a few of 2^28 rows
    assert abs(loss.item() - 1) <= 2.0 ** -17
    d = tw.bl_route_backward(logits, index, dweight, renorm=False, coef=coef, dloss=torch.ones_like(loss), out_dtype=torch.float32)
    ih = index[-37:].cpu().numpy()
    check_gradient(d[-37:], lh, ih, "softmax", False, 1.0, "fp32", dweight=np.ones((37, 1), np.float32), coef=host(coef), dloss=np.ones(1))
    assert torch.equal(d[:4096], d[4096:8192]) and torch.equal(d[:4096], d[(1 << 27):(1 << 27) + 4096])
