"""The router's choice where FP32 cannot make it: every decision that 64 bits settle is the one of 64
bits, for scores of any size.  (The hardware's exponential is off by some 1.2 |x| units of its last
place, so that scores of logits far below 0 are less exact than those next to 1.)"""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from route_harness import choice

pytestmark = pytest.mark.gpu
SOFT, SIG = lib.GEMM_SCORE_SOFTMAX, lib.GEMM_SCORE_SIGMOID


def settled(x, k, score, bias=None, groups=1, kept=1, top=1, share=0.9):
    """The library's choice is that of 64 bits wherever those settle it, in most tokens."""
    x = np.asarray(x, dtype=np.float32)
    b = None if bias is None else np.asarray(bias, dtype=np.float32)
    chosen, _ = lib.route(torch.from_numpy(x).cuda(), k, score=score, groups=groups, groups_kept=kept,
                          group_top=top, bias=None if b is None else torch.from_numpy(b).cuda())
    ids, sure = choice(x.astype(np.float64), k, score, None if b is None else b.astype(np.float64),
                       groups, kept, top)
    assert sure.mean() >= share, sure.mean()
    off = (chosen.cpu().numpy() != ids).any(1) & sure
    assert not off.any(), f"{int(off.sum())} of {int(sure.sum())} tokens"


def moved(x, units):
    """FP32 values so many units of their last place further."""
    return (x.astype(np.float32).view(np.int32) + units.astype(np.int32)).view(np.float32)


@pytest.mark.parametrize("center", [0, -5, -10, -20, -40, -60, -80])
@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (64, 8, 2), (96, 6, 3)])
@pytest.mark.parametrize("biased", [True, False])
def test_groups_of_small_scores(center, experts, groups, kept, biased):
    """Groups of the same logits up to a few units of their last place, each in an order of its own."""
    rng = np.random.default_rng([experts, -center])
    T, size = 4000, experts // groups
    base = (center + rng.standard_normal((T, 1, size))).astype(np.float32)
    x = np.repeat(base, groups, 1)
    x = moved(x, rng.integers(-40, 41, x.shape) * (rng.random(x.shape) < 0.5))
    x = rng.permuted(x, axis=2).reshape(T, experts)
    settled(x, min(6, size), SIG, np.zeros(experts) if biased else None, groups, kept, 2)
    settled(x, min(6, size), SIG, np.zeros(experts) if biased else None, groups, kept, 1)


@pytest.mark.parametrize("center", [0, -5, -10, -20, -40, -60, -80])
@pytest.mark.parametrize("experts,k", [(256, 8), (64, 6), (33, 3)])
def test_biases_of_the_scores_size(center, experts, k):
    """s + b nearly the same for all: b is a constant of the largest score's size less s, rounded to
    FP32 -- exactly for the row that it is made from, to some units for the others."""
    rng = np.random.default_rng([experts, -center])
    x0 = (center + rng.standard_normal(experts)).astype(np.float32)
    s = 1 / (1 + np.exp(-x0.astype(np.float64)))
    for times in (1.5, 4.0):
        bias = (times * s.max() - s).astype(np.float32)
        x = moved(np.repeat(x0[None], 2000, 0), rng.integers(-30, 31, (2000, experts)))
        settled(x, k, SIG, bias)
        if experts % 8 == 0:
            settled(x, min(k, 2 * experts // 8), SIG, bias, 8, 2, 2)


@pytest.mark.parametrize("depth", [5, 20, 40, 60, 80])
@pytest.mark.parametrize("experts,k", [(256, 8), (64, 6)])
def test_softmax_scores_far_below_a_masked_one(depth, experts, k):
    """The largest logits belong to experts that the bias masks: the scores of the others are small, and
    their biases too."""
    rng = np.random.default_rng([experts, depth])
    x0 = (rng.standard_normal(experts) - depth).astype(np.float32)
    x0[5], x0[17] = 0.5, 1.0
    e = np.exp(x0.astype(np.float64) - 1.0)
    s = e / e.sum()
    few = np.ones(experts, dtype=bool)
    few[[5, 17]] = False
    bias = (1.5 * s[few].max() - s).astype(np.float32)
    bias[[5, 17]] = -np.inf
    x = moved(np.repeat(x0[None], 2000, 0), rng.integers(-30, 31, (2000, experts)))
    settled(x, k, SOFT, bias)
    settled(x, k, SOFT, bias, 8, 3, 2)


@pytest.mark.parametrize("biased", [True, False])
def test_scores_below_fp32(biased):
    """Sigmoid scores at and below 2^-126, where FP32 results are cut to 0."""
    rng = np.random.default_rng(1)
    for center in (-85.0, -88.0, -95.0, -103.0, -200.0):
        x = center + rng.standard_normal((3000, 64)) * 1.5
        bias = np.zeros(64) if biased else None
        settled(x, 6, SIG, bias)
        settled(x, 6, SIG, bias, 8, 3, 2)
        settled(x, 6, SIG, bias, 8, 3, 1)
    if biased:  # some scores are 0 in FP32, some biases below 2^-126
        x = -87.0 + rng.standard_normal((3000, 64))
        settled(x, 6, SIG, rng.random(64) * 2e-38, 8, 3, 2)
        settled(x, 6, SIG, rng.random(64) * 2e-38)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (256, 32, 7), (160, 8, 3), (64, 2, 1)])
def test_every_settled_token(score, biased, top, experts, groups, kept):
    """Ordinary logits, some groups equal or a few units apart: no token is allowed to be wrong."""
    rng = np.random.default_rng([experts, groups, top])
    T, size = 4000, experts // groups
    base = rng.standard_normal((T, 1, size)).astype(np.float32) * 1.5
    x = np.repeat(base, groups, 1)
    x = moved(x, rng.integers(-3, 4, x.shape) * (rng.random(x.shape) < 0.3))
    bias = np.tile(0.1 * rng.standard_normal(size), groups) if biased else None
    if not biased:
        x = rng.permuted(x, axis=2)
    x[::9] = base[::9, :, :]
    x[::11, 1::2] = rng.standard_normal((len(x[::11]), groups // 2, size)).astype(np.float32)
    x = x.reshape(T, experts)
    settled(x, min(6, size), score, bias, groups, kept, top)
    settled(x, min(6, size), score, bias)
