"""An expert whose bias is -infinity is out of the router's choice, also where its logit is a NaN or
an infinity: with both scores, with and without groups, in each way the choice is made (in FP32,
groups or candidates compared again in 64 bits, the whole token in 64 bits)."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import f64
from mixture_harness import stored
from route_harness import choice

pytestmark = pytest.mark.gpu
SOFT, SIG = lib.GEMM_SCORE_SOFTMAX, lib.GEMM_SCORE_SIGMOID
INF = float("inf")


def run(x, k, score, bias, groups=1, kept=1, top=1, dtype="f32", renorm=True):
    logits = stored(x, dtype)
    chosen, w = lib.route(logits, k, score=score, bias=torch.from_numpy(bias.astype(np.float32)).cuda(),
                          groups=groups, groups_kept=kept, group_top=top, renormalize=renorm)
    ids, sure = choice(f64(logits), k, score, bias.astype(np.float32).astype(np.float64), groups, kept, top)
    assert sure.mean() > 0.9
    assert np.array_equal(chosen.cpu().numpy()[sure], ids[sure])
    assert not np.isin(chosen.cpu().numpy(), np.flatnonzero(bias == -INF)).any()
    assert (w[chosen < 0] == 0).all()
    return chosen, w


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 2), (4, 2, 1), (8, 3, 2)])
@pytest.mark.parametrize("value", [float("nan"), INF])
def test_a_masked_sigmoid_score_is_not_seen(dtype, renorm, groups, kept, top, value):
    """The garbage of masked experts leaves the others' choice and weights as if it were a 0."""
    rng = np.random.default_rng([groups, top])
    for E, k in ((32, 5), (64, 32), (96, 8), (1000, 8)):
        x = rng.standard_normal((40, E)) * 1.5
        bias = rng.standard_normal(E) * 0.1
        off = rng.permutation(E)[:E // 5 + 1]
        bias[off] = -INF
        clean = x.copy()
        x[:, off[0]] = value
        x[1, off] = value
        x[2, off[1:]] = value
        clean[:, off] = 0.0
        kc = min(k, E // groups * kept)
        got = run(x, kc, SIG, bias, groups, kept, top, dtype, renorm)
        want = run(clean, kc, SIG, bias, groups, kept, top, dtype, renorm)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.isfinite(got[1]).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
@pytest.mark.parametrize("value", [float("nan"), INF])
def test_softmax_scores_of_a_row_with_a_nan(renorm, groups, kept, top, value):
    """Every score of the row is a NaN, and so are its weights; the experts in the choice come by their
    indices, those that the bias masks do not come at all."""
    rng = np.random.default_rng(groups)
    x = rng.standard_normal((8, 32))
    bias = rng.standard_normal(32) * 0.1
    bias[[0, 1, 5, 9, 30]] = -INF
    x[2, 5] = value   # masked
    x[3, 7] = value   # not masked
    x[4, [0, 9]] = value
    x[5] = value
    chosen, w = run(x, 6, SOFT, bias, groups, kept, top, "f32", renorm)
    left = [e for e in range(32) if bias[e] != -INF]
    for t in (2, 3, 4, 5):
        assert chosen[t].tolist() == left[:6]
        assert torch.isnan(w[t]).all()
    for t in (0, 1, 6, 7):
        assert torch.isfinite(w[t]).all()


@pytest.mark.parametrize("score", [SOFT, SIG])
def test_everything_is_masked(score):
    x = np.random.default_rng(0).standard_normal((6, 24))
    x[1, 3], x[2] = np.nan, np.nan
    x[3, 5] = INF
    chosen, w = run(x, 4, score, np.full(24, -INF))
    assert (chosen == -1).all() and (w == 0).all()
    bias = np.full(24, -INF)
    bias[17] = 0.25
    chosen, w = run(x, 4, score, bias)
    assert (chosen[:, 0] == 17).all() and (chosen[:, 1:] == -1).all() and (w[:, 1:] == 0).all()
    nan = [2] if score == SIG else [1, 2, 3]
    assert torch.isnan(w[nan, 0]).all()
    assert (w[[t for t in range(6) if t not in nan], 0] == 1).all()


@pytest.mark.parametrize("k,top", [(6, 2), (6, 1), (20, 2)])
@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (64, 4, 2), (1024, 16, 3)])
def test_masked_nans_where_64_bits_decide(k, top, experts, groups, kept):
    """Equal and nearly equal values: groups, candidates or whole tokens are computed again."""
    rng = np.random.default_rng([experts, k, top])
    T, size = 200, experts // groups
    base = rng.standard_normal((T, 1, size)).astype(np.float32)
    units = rng.integers(-3, 4, (T, groups, size)) * (rng.random((T, groups, size)) < 0.3)
    x = (np.repeat(base, groups, 1).view(np.int32) + units.astype(np.int32)).view(np.float32)
    x[::5] = 0.25  # a row of equal logits: more candidates than lanes
    x = x.reshape(T, experts).astype(np.float64)
    bias = np.tile(0.1 * rng.standard_normal(size), groups)
    bias[rng.permutation(experts)[:experts // 6]] = -INF
    bias[::size] = -INF
    for e in np.flatnonzero(bias == -INF):
        x[rng.random(T) < 0.5, e] = np.nan
    run(x, k, SIG, bias, groups, kept, top)
    run(x, k, SIG, bias)
    bias[bias != -INF] = 0.0  # (of equal logits every candidate is a tie)
    run(x, k, SIG, bias, groups, kept, top)
    run(x, k, SIG, bias)
