"""Scores far below the largest: gradients of the router where what was chosen has next to no score,
as a choice by bias or by another routing leaves it, and the balance loss of logits far apart.

Bounds. u = 2^-24 is half a unit of fp32. An exponential errs by two units, and by u |l - max| of its
argument's rounding; results below 2^-126 are multiples of 2^-149, off by at most one each for the
exponential and for its product with 1 / sum."""
import numpy as np
import pytest
import torch

import oracle.adapters as oa
import ternary_weight_linear_amd as tw
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu

u, step = 2.0 ** -24, 2.0 ** -149


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def host(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("E,k", [(20, 1), (64, 2), (128, 3), (300, 4), (600, 2), (2048, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_renormalised_weights_of_scores_that_fp32_hardly_holds(E, k, score):
    """Every row's experts are even but for the chosen ones, whose scores lie around and below 2^-126. Their
    weights are those of any other row, and so is their gradient."""
    say("route tiny scores", E, k, score)
    g = np.random.default_rng(E + k)
    depth = np.concatenate([np.linspace(80, 93, 40), [87.2, 87.33, 87.34, 88.0, 88.5, 88.7]])
    if score == "sigmoid":
        depth = np.minimum(depth, 88.0)                        # below, the weights themselves are 0
    M = depth.size
    lh = np.zeros((M, E), np.float32)
    index = np.stack([g.permutation(E)[:k] for _ in range(M)]).astype(np.int32)
    chosen = (-depth[:, None] + g.random((M, k)) * 0.5).astype(np.float32)
    np.put_along_axis(lh, index, chosen, 1)
    dweight = g.standard_normal((M, k)).astype(np.float32)
    d = host(tw.bl_route_backward(gpu(lh), gpu(index), gpu(dweight), score=score, renorm=True, factor=1.5))
    assert np.isfinite(d).all()
    ref, mag = oa.route_backward(lh, index, score, True, 1.5, dweight)
    p = oa.scores(lh, score)[0]
    least = np.take_along_axis(p, index, 1).min(1)
    # a slot's share of their sum: each score's error and its sum's, again in the mean over the slots, in
    # products and quotients of a few roundings each
    each = (2 * 94 + E / 8 + 40) * u + 2 * step / least
    assert np.all(np.abs(d - ref) <= 6 * each[:, None] * mag + step)


@pytest.mark.parametrize("E", [6, 64, 600])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_one_expert_far_above_the_others(E, score):
    """A logit of 3e38: softmax scores are one and zeros exactly, so the loss is that expert's
    coefficient and no logit has a gradient. Sigmoid scores are one there, and one half and less elsewhere."""
    say("route far apart", E, score)
    g = np.random.default_rng(E)
    lh = (-np.abs(g.standard_normal((1, E)))).astype(np.float32)
    lh[0, 0] = 3e38
    index = np.array([[0, 1, E - 1]], np.int32)
    loss, count, coef = tw.bl_route_balance(gpu(lh), gpu(index), score=score)
    rloss, rcount, rcoef = oa.balance(lh, index, score)
    assert np.array_equal(count.cpu().numpy(), rcount) and np.all(np.abs(host(coef) - rcoef) <= 2 * u * rcoef)
    dweight = g.standard_normal((1, 3)).astype(np.float32)
    one = torch.ones(1, device=DEV)
    for renorm in (True, False):
        d = host(tw.bl_route_backward(gpu(lh), gpu(index), gpu(dweight), score=score, renorm=renorm, coef=coef, dloss=one))
        ref, mag = oa.route_backward(lh, index, score, renorm, 1.0, dweight, host(coef), np.ones(1))
        if score == "softmax":
            assert loss.item() == coef[0, 0].item() and not d.any() and not ref.any()
        else:
            # exponentials of at most 5 in size, sums of E terms in chains of E / 16 + 4
            bound = (2 * 5 + E / 8 + 40) * u
            assert abs(loss.item() - rloss[0]) <= bound * rloss[0] and np.all(np.abs(d - ref) <= 2 * bound * mag + step)


def test_falling_offsets_write_nothing_outside_the_buffers():
    """Offsets that fall are outside the contract: any numbers may come back, inside the outputs and the workspace,
    which stand here between guards."""
    say("route falling offsets, guarded")
    M, E, k, S = 3000, 40, 2, 7
    g = np.random.default_rng(7)
    logits, index = gpu(g.standard_normal((M, E)).astype(np.float32)), gpu(g.integers(-1, E, (M, k)).astype(np.int32))
    dloss, guard = torch.ones(S, device=DEV), 1 << 16
    sizes = [S * 4, S * E * 4, S * E * 4, tw._lib.bl_route_balance_workspace_bytes(M, E, S), M * E * 4]
    rows = [-5, 0, 1, 400, 1500, 2999, 3000, 3001, 2 ** 31 - 1, -2 ** 31]
    for turn in range(40):
        offsets = gpu(g.choice(rows, S + 1).astype(np.int32))
        at, room = [], torch.full((sum(-(-n // 256) * 256 + guard for n in sizes) + guard,), 0xA5, dtype=torch.uint8, device=DEV)
        kept = torch.ones(room.numel(), dtype=torch.bool, device=DEV)
        where = guard
        for n in sizes:
            at.append(room.data_ptr() + where)
            kept[where:where + n] = False
            where += -(-n // 256) * 256 + guard
        for score in (0, 1):
            assert tw._lib.bl_route_balance(logits.data_ptr(), 2, M, E, E, index.data_ptr(), k, score, offsets.data_ptr(), S, at[0], at[1], at[2],
                                            at[3], sizes[3], tw._stream(logits.device)) == 0
            assert tw._lib.bl_route_backward(logits.data_ptr(), 2, M, E, E, index.data_ptr(), k, score, None, 0, 1.0, at[2], dloss.data_ptr(),
                                             offsets.data_ptr(), S, at[4], 2, E, tw._stream(logits.device)) == 0
        torch.cuda.synchronize()
        assert torch.all(room[kept] == 0xA5), offsets.tolist()
