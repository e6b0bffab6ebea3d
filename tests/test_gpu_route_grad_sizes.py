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
