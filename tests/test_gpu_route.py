"""The router against its definition in 64 bits: the choice is exact, ties and
masks included; weights and gradients within derived bounds."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import f64
from mixture_harness import check, route_grad_ref, route_ref, rounding, stored

pytestmark = pytest.mark.gpu
SOFT, SIG = lib.GEMM_SCORE_SOFTMAX, lib.GEMM_SCORE_SIGMOID


def weight_tol(w, x, scale, renorm):
    """exp(x - m) in FP32: x - m is rounded (2^-24 |x - m| of the result; |x - m| is at most the
    row's spread), expf is off by 2 units, the sum of at most 1024 positive terms by 37 roundings (32 of
    a lane, 5 across), division and scale by 2."""
    finite = np.where(np.isfinite(x), x, 0.0)
    spread = finite.max(-1, keepdims=True) - finite.min(-1, keepdims=True)
    return np.abs(w) * (np.minimum(spread, 110.0) + 50) * 2.0 ** -23 + 2.0 ** -125 * max(scale, 1.0)


def run(x, dtype, k, score, bias=None, groups=1, kept=1, top=1, renorm=True, scale=1.0, extra=0):
    logits = stored(x, dtype, extra)
    b = torch.tensor(bias, dtype=torch.float32).cuda() if bias is not None else None
    chosen, w = lib.route(logits, k, score=score, bias=b, groups=groups, groups_kept=kept,
                          group_top=top, renormalize=renorm, scale=scale)
    assert lib.gemm_last_kernel() == "route"
    xd = f64(logits)
    bd = f64(b) if b is not None else None
    ids, ref = route_ref(xd, k, score, bd, groups, kept, top, renorm, scale)
    assert np.array_equal(chosen.cpu().numpy(), ids)
    check(w, ref, weight_tol(ref, xd, scale, renorm), "weights")
    return logits, chosen, w


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 64, 8), (3, 5, 5), (7, 31, 3), (5, 33, 4),
                                              (9, 64, 6), (130, 128, 8), (66, 160, 6), (37, 256, 8),
                                              (3, 1000, 32), (2, 1024, 7), (4, 512, 32), (5, 77, 1)])
def test_choice_and_weights(dtype, score, tokens, experts, k):
    rng = np.random.default_rng([tokens, experts, k])
    x = rng.standard_normal((tokens, experts)) * 2
    run(x, dtype, k, score, renorm=True, scale=2.5)
    run(x, dtype, k, score, renorm=False, extra=3)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("experts,groups,kept,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 8),
                                                   (12, 4, 2, 6), (33, 3, 1, 11), (32, 32, 7, 7),
                                                   (63, 7, 7, 9), (1024, 16, 2, 32), (20, 10, 1, 2)])
def test_groups(score, top, biased, experts, groups, kept, k):
    rng = np.random.default_rng([experts, groups, top])
    x = rng.standard_normal((45, experts)) * 1.5
    bias = rng.standard_normal(experts) * 0.1 if biased else None
    for dtype in ("f32", "bf16"):
        run(x, dtype, k, score, bias, groups, kept, top, scale=2.5)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_ties_go_to_the_lowest_index(score, biased, groups, kept):
    rng = np.random.default_rng(5)
    x = rng.integers(-1, 2, (60, 64)).astype(float)
    x[0] = 0.0  # all equal
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[2, 1::2] = 0.0
    bias = rng.integers(0, 2, 64) * 0.25 if biased else None
    run(x, "f32", 12, score, bias, groups, kept, 2)
    run(x, "bf16", 12, score, bias, groups, kept, 1)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_values_that_fp32_cannot_tell_apart(dtype):
    """Scores next to 1, and sums with a bias closer than FP32 holds: the order is that of 64 bits."""
    rng = np.random.default_rng(6)
    T, E = 40, 96
    x = 17 + rng.permuted(np.arange(E)[None].repeat(T, 0) / 16.0, axis=1)  # 1 - s from 4e-8 down
    bias = np.zeros(E)
    run(x, dtype, 8, SIG, bias, renorm=False)
    run(x, dtype, 8, SIG, bias, groups=4, kept=2, top=2)
    run(x, dtype, 8, SIG, None, groups=4, kept=2, top=2)  # group sums next to 2
    # s + b nearly constant: b = -s(x) rounded to FP32, logits of 1e-4 apart
    x = 0.3 + rng.standard_normal((T, E)) * 1e-4
    x[:] = x[0]
    s = 1 / (1 + np.exp(-x[0].astype(np.float32).astype(np.float64)))
    run(x, "f32", 16, SIG, (1 - s).astype(np.float32))
    # softmax scores of one size with a large bias
    x = rng.standard_normal((T, E)) * 1e-5
    run(x, "f32", 16, SOFT, np.full(E, 3.0))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_masked_experts(score, biased, groups, kept, top):
    rng = np.random.default_rng(7)
    x = rng.standard_normal((30, 32))
    x[rng.random(x.shape) < 0.5] = -np.inf
    x[0] = -np.inf  # nothing left
    x[1, 1:] = -np.inf  # one left
    x[2, :31] = -np.inf
    x[3, 8:] = -np.inf  # one group left
    bias = rng.standard_normal(32) if biased else None
    if biased:
        bias[5] = -np.inf
    for dtype in ("f32", "f16"):
        _, chosen, w = run(x, dtype, 9, score, bias, groups, kept, top)
        assert (chosen[0] == -1).all() and (w[0] == 0).all()
        run(x, dtype, 9, score, bias, groups, kept, top, renorm=False)


@pytest.mark.parametrize("dtype,lowest", [("f32", -3.4028234663852886e38), ("f16", -65504.0),
                                          ("bf16", -3.3895313892515355e38)])
@pytest.mark.parametrize("score", [SOFT, SIG])
def test_the_types_lowest_value_is_no_mask(dtype, lowest, score):
    rng = np.random.default_rng(8)
    x = rng.standard_normal((6, 40))
    x[0] = lowest
    x[1, 3:] = lowest
    x[2, ::2] = lowest
    _, chosen, w = run(x, dtype, 6, score)
    assert (chosen >= 0).all() and torch.isfinite(w).all()
    run(x, dtype, 6, score, np.zeros(40), renorm=False)
    run(np.full((2, 40), -200.0) - np.arange(40) / 4, dtype, 6, score)  # scores below FP32


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("groups", [1, 4])
def test_nans_and_infinities_stay_in_their_row(score, groups):
    rng = np.random.default_rng(9)
    x = rng.standard_normal((6, 32))
    clean = x.copy()
    x[1, 7] = np.nan
    x[2, 9] = np.inf
    x[3] = np.nan
    x[4, [3, 20]] = [np.inf, np.nan]
    for bias in (None, np.zeros(32)):
        b = None if bias is None else torch.zeros(32, device="cuda")
        a = dict(score=score, bias=b, groups=groups, groups_kept=2, group_top=2)
        chosen, w = lib.route(stored(x, "f32"), 5, **a)
        same, ws = lib.route(stored(clean, "f32"), 5, **a)
        for t in (0, 5):
            assert torch.equal(chosen[t], same[t]) and torch.equal(w[t], ws[t])
        assert ((chosen >= 0) & (chosen < 32)).all()
        assert all(len(set(r.tolist())) == 5 for r in chosen)
        # a NaN is chosen first, and shows
        assert torch.isnan(w[1, 0])
        if bias is not None and score == SOFT:  # every s of the row is a NaN, and so is every c: ties
            assert chosen[1, 0] == 0 and chosen[2, 0] == 0
            continue
        assert chosen[1, 0] == 7 and chosen[2, 0] == 9
        if groups == 1:
            assert chosen[3].tolist() == [0, 1, 2, 3, 4]
            assert chosen[4, :2].tolist() == [20, 3]
        assert torch.isnan(w[3]).all()


def test_every_nan_is_the_same():
    """NaNs of either sign and any payload are chosen first, by their numbers."""
    bits = np.array([0x7f800001, 0xff800001, 0x7fc00000, 0xffffffff, 0xffc12345], dtype=np.uint32)
    x = np.zeros((5, 40), dtype=np.float32)
    x[:, 7:40:8] = bits.view(np.float32)[:5][None].repeat(5, 0)[:, :5]
    chosen, w = lib.route(torch.from_numpy(x).cuda(), 6, score=SIG, renormalize=False)
    assert chosen.cpu().tolist() == [[7, 15, 23, 31, 39, 0]] * 5
    assert torch.isnan(w[:, :5]).all() and (w[:, 5] == 0.5).all()


def test_many_tokens_and_every_row_once():
    """More tokens than one pass of the grid at once, the last ones too."""
    T, E, k = 70001, 16, 3
    x = torch.randn(T, E, device="cuda")
    chosen, w = lib.route(x, k)
    v, i = torch.sort(x, dim=1, descending=True, stable=True)
    assert torch.equal(chosen.long(), i[:, :k])
    ref = torch.softmax(v[:, :k].double(), 1)
    assert (w.double() - ref).abs().max() < 60 * 2.0 ** -23


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 64, 8), (6, 5, 5), (13, 33, 4), (66, 160, 6),
                                              (9, 256, 8), (2, 1000, 32), (5, 77, 1), (3, 1024, 8)])
def test_gradient(dtype, score, renorm, tokens, experts, k):
    rng = np.random.default_rng([tokens, experts, k])
    logits = stored(rng.standard_normal((tokens, experts)) * 2, dtype, extra=5)
    chosen, _ = lib.route(logits, k, score=score)
    ids = chosen.cpu().numpy()
    dw = torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).cuda()
    x = f64(logits)
    ref = route_grad_ref(x, ids, f64(dw), score, renorm, 2.5)
    # every term is a product of scores (each off by (spread + 50) 2^-23, spread < 20) and dw, summed
    # over at most 32: twice 80 units and 32 roundings of scale * sum |dw|, in proportion to the
    # largest score of the term
    size = 2.5 * np.abs(f64(dw)).sum(1, keepdims=True)
    tol = 200 * 2.0 ** -23 * size + rounding(dtype, ref)
    kw = dict(score=score, renormalize=renorm, scale=2.5)
    got = lib.route_grad(logits, chosen, dw, **kw)
    assert lib.gemm_last_kernel() == "route_grad"
    check(got, ref, tol)
    # into a padded matrix, and over the logits themselves
    out = stored(np.zeros((tokens, experts)), dtype, extra=3, fill=7.0)
    assert torch.equal(lib.route_grad(logits, chosen, dw, out=out, **kw), got)
    base = out._base if out._base is not None else out
    assert (base[:, experts:] == 7.0).all()
    over = logits.clone()
    assert torch.equal(lib.route_grad(over, chosen, dw, out=over, **kw), got)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the weights in 64 bits, the choice fixed: their error is h^2 times a third
    derivative (scores and ratios of them: below 10) and 2^-52 / h."""
    rng = np.random.default_rng(3)
    T, E, k, h = 4, 12, 3, 1e-4
    x = rng.standard_normal((T, E)).astype(np.float32).astype(np.float64)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    ids, _ = route_ref(x, k, score, None, 1, 1, 1, renorm, 1.5)

    def value(y):
        from mixture_harness import scores
        w = np.take_along_axis(scores(y, score), ids, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return 1.5 * (w * dw).sum(1)

    ref = np.zeros((T, E))
    for e in range(E):
        up, down = x.copy(), x.copy()
        up[:, e] += h
        down[:, e] -= h
        ref[:, e] = (value(up) - value(down)) / (2 * h)
    got = lib.route_grad(torch.from_numpy(x.astype(np.float32)).cuda(),
                         torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(dw).cuda(),
                         score=score, renormalize=renorm, scale=1.5)
    size = 1.5 * np.abs(dw).sum(1, keepdims=True)
    check(got, ref, size * (10 * h * h + 1e-10 + 200 * 2.0 ** -23))


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("experts,groups,kept", [(256, 8, 4), (256, 16, 5), (256, 32, 7), (160, 8, 3), (64, 2, 1)])
def test_groups_that_fp32_cannot_tell_apart(score, biased, top, experts, groups, kept):
    """Groups of the same logits, each in an order of its own, some a few units apart or equal."""
    rng = np.random.default_rng([experts, groups, top])
    T, size = 300, experts // groups
    base = rng.standard_normal((T, 1, size)).astype(np.float32) * 1.5
    x = np.repeat(base, groups, 1)
    units = rng.integers(-3, 4, x.shape) * (rng.random(x.shape) < 0.3)
    x = (x.view(np.int32) + units.astype(np.int32)).view(np.float32)
    bias = np.tile(0.1 * rng.standard_normal(size), groups).astype(np.float32) if biased else None
    if not biased:
        x = rng.permuted(x, axis=2)
    x[::9] = base[::9, :, :]  # equal groups
    x[::11, 1::2] = rng.standard_normal((len(x[::11]), groups // 2, size)).astype(np.float32)
    x = x.reshape(T, experts)
    for g, n in ((groups, kept), (1, 1)):  # (and by themselves)
        chosen, _ = lib.route(torch.from_numpy(x).cuda(), min(6, size), score=score,
                              bias=torch.from_numpy(bias).cuda() if biased else None, groups=g,
                              groups_kept=n, group_top=top)
        ids, _ = route_ref(x.astype(np.float64), min(6, size), score,
                           None if bias is None else bias.astype(np.float64), g, n, top, True, 1.0)
        off = (chosen.cpu().numpy() != ids).any(1)
        # (64 bits round too: sums of two scores below 2 that are within 2^-50 may go either way)
        assert off.sum() <= T // 100, off.sum()


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("experts", [1, 28, 64])
def test_a_single_expert_takes_all(dtype, score, experts):
    """Renormalised, one expert's weight is 1 whatever its logit, and the gradient 0: exactly."""
    rng = np.random.default_rng(experts)
    logits = stored(rng.standard_normal((1000, experts)) * 3, dtype)
    dw = torch.from_numpy(rng.standard_normal((1000, 1)).astype(np.float32)).cuda()
    chosen, w = lib.route(logits, 1, score=score, scale=2.5)
    assert (w == 2.5).all()
    assert (lib.route_grad(logits, chosen, dw, score=score, scale=2.5) == 0).all()
    if experts < 4:
        return
    more = torch.full((1000, 4), -1, dtype=torch.int32, device="cuda")
    more[:, 2] = chosen[:, 0]
    assert (lib.route_grad(logits, more, dw.expand(1000, 4).contiguous(), score=score) == 0).all()


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("renorm", [True, False])
def test_one_expert_named_many_times(score, renorm):
    """All 32 places name two experts: the sums are the formula's, and the same bits every time."""
    rng = np.random.default_rng(8)
    x = rng.standard_normal((40, 33))
    ids = np.where(rng.random((40, 32)) < 0.5, 3, 7)
    dw = rng.standard_normal((40, 32)).astype(np.float32)
    args = (stored(x, "f32"), torch.from_numpy(ids.astype(np.int32)).cuda(), torch.from_numpy(dw).cuda())
    got = lib.route_grad(*args, score=score, renormalize=renorm)
    ref = route_grad_ref(f64(args[0]), ids, dw.astype(np.float64), score, renorm, 1.0)
    check(got, ref, 200 * 2.0 ** -23 * np.abs(dw).sum(1, keepdims=True))
    for _ in range(5):
        assert torch.equal(lib.route_grad(*args, score=score, renormalize=renorm), got)


def test_gradient_of_dropped_repeated_and_masked_experts():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((5, 16))
    x[2, 4:] = -np.inf
    ids = np.array([[3, -1, 5], [-1, -1, -1], [0, 2, 1], [7, 7, 2], [16, 1 << 30, 4]])
    dw = rng.standard_normal((5, 3)).astype(np.float32)
    dw[0, 1] = dw[1, 0] = dw[4, 0] = np.nan  # of places without an expert: not read as numbers
    clean = np.where(np.isnan(dw), 0, dw).astype(np.float64)
    for score in (SOFT, SIG):
        for renorm in (True, False):
            ref = route_grad_ref(x, ids, clean, score, renorm, 1.0)
            got = lib.route_grad(stored(x, "f32"), torch.from_numpy(ids.astype(np.int32)).cuda(),
                                 torch.from_numpy(dw).cuda(), score=score, renormalize=renorm)
            check(got, ref, 200 * 2.0 ** -23 * np.abs(clean).sum(1, keepdims=True) + 1e-30)
            assert (got[1] == 0).all()


def test_streams_graphs_and_two_calls_at_once():
    x = [torch.randn(300, 64, device="cuda") for _ in range(2)]
    want = [lib.route(t, 4) for t in x]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [lib.route(t, 4, stream=s) for t, s in zip(x, side)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    dw = torch.randn(300, 4, device="cuda")
    ref = lib.route_grad(x[0], want[0][0], dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chosen, weights = lib.route(x[0], 4)
        d = lib.route_grad(x[0], chosen, dw)
    for _ in range(2):
        chosen.zero_()
        graph.replay()
        assert torch.equal(chosen, want[0][0]) and torch.equal(weights, want[0][1])
        assert torch.equal(d, ref)
    x[0].copy_(x[1])
    graph.replay()
    assert torch.equal(chosen, want[1][0])


def test_helper_refusals_on_the_device():
    x = torch.randn(4, 8, device="cuda")
    for bad in (dict(k=0), dict(k=9), dict(k=2, groups=3), dict(k=2, score=5),
                dict(k=2, groups=2, groups_kept=3), dict(k=2, groups=2, group_top=3)):
        with pytest.raises(lib.GemmError):
            lib.route(x, **bad)
    with pytest.raises(lib.GemmError):
        lib.route(torch.randn(4, 1025, device="cuda"), 2)
    with pytest.raises(ValueError):
        lib.route(x, 2, bias=torch.zeros(8))  # on the CPU


def test_offsets_past_32_bits():
    """Rows more than 2^31 elements into the logits."""
    T, E = 3, 32
    pitch = (1 << 30) + 8
    big = torch.empty(2 * pitch + E, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, E), (pitch, 1))
    x.copy_(torch.randn(T, E))
    small = x.clone()
    c, w = lib.route(x, 4)
    cs, ws = lib.route(small, 4)
    assert torch.equal(c, cs) and torch.equal(w, ws)
    dw = torch.randn(T, 4, device="cuda")
    assert torch.equal(lib.route_grad(x, c, dw, out=x), lib.route_grad(small, cs, dw))
