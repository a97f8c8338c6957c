"""gemm_lora against its definition in 64 bits: types, orders, ranks, rows
without an adapter, rows in any order, adapters with special values."""
import itertools

import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import (SENTINEL, TORCH, assert_close, done, draw, lora_ref, offsets_of,
                             padded, wgrad_ref)

pytestmark = pytest.mark.gpu


def operands(rng, M, K, N, rank, n, dtype, order, pad=8, dist="normal"):
    k = max(K, 1) ** -0.5
    X = padded(draw(rng, (M, K), dtype, dist), pad)
    if order[0]:
        W = padded(draw(rng, (N, K), dtype, dist, k), pad).t()
    else:
        W = padded(draw(rng, (K, N), dtype, dist, k), pad)
    if order[1]:
        LA = padded(draw(rng, (n, rank, K), dtype, dist, k), pad).transpose(1, 2)
    else:
        LA = padded(draw(rng, (n, K, rank), dtype, dist, k), pad)
    if order[2]:
        LB = padded(draw(rng, (n, N, rank), dtype, dist, 0.5), pad).transpose(1, 2)
    else:
        LB = padded(draw(rng, (n, rank, N), dtype, dist, 0.5), pad)
    return X, W, LA, LB


def run(rng, M, K, N, rank, n, dtype, out, order=(1, 1, 1), ids=None, scale=True, bias=False,
        act=0, pad=8, pad_d=0, dist="normal"):
    X, W, LA, LB = operands(rng, M, K, N, rank, n, dtype, order, pad, dist)
    if ids is None:
        ids = rng.integers(-1, n, M)
    ids = torch.from_numpy(np.asarray(ids).astype(np.int32)).cuda()
    s = torch.from_numpy((rng.random(n) + 0.5).astype(np.float32)).cuda() if scale else None
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda() if bias else None
    buf = torch.full((M + 1, N + pad_d), SENTINEL, dtype=TORCH[out], device="cuda")
    D = buf[:M, :N]
    lib.gemm_lora(X, W, LA, LB, ids, scale=s, bias=b, activation=act, out=D)
    name = lib.gemm_last_kernel()
    done()
    ref, tol = lora_ref(X, W, LA, LB, ids, s, b, act, dtype, out)
    assert_close(D, ref, tol, out, f"{name} {dtype} M {M} K {K} N {N} rank {rank} n {n} {order}")
    left = buf.clone()
    left[:M, :N] = SENTINEL
    assert bool((left == SENTINEL).all()), "a store outside D"
    return name


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                       ("f16", "f32")])
@pytest.mark.parametrize("M,K,N,rank,n", [
    (1, 256, 256, 16, 4), (2, 64, 8, 8, 1), (7, 1000, 520, 16, 3), (64, 512, 1030, 16, 48),
    (128, 328, 264, 64, 5), (129, 72, 257, 32, 200), (300, 200, 136, 24, 7), (500, 264, 640, 128, 3),
    (33, 136, 200, 1, 6)])
def test_lora_shapes(dtype, out, M, K, N, rank, n):
    run(np.random.default_rng(M + K), M, K, N, rank, n, dtype, out, pad_d=8)


@pytest.mark.parametrize("order", list(itertools.product([0, 1], repeat=3)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [5, 200])
def test_lora_orders(order, dtype, M):
    run(np.random.default_rng(M), M, 264, 392, 16, 9, dtype, "f32", order=order)
    run(np.random.default_rng(M + 1), M, 200, 136, 40, 3, dtype, dtype, order=order, pad_d=3)


@pytest.mark.parametrize("ids", ["none", "one", "runs", "distinct", "outside"])
@pytest.mark.parametrize("M", [1, 40, 260])
def test_lora_row_patterns(ids, M):
    rng = np.random.default_rng(M)
    n = 300
    pattern = {"none": np.full(M, -1), "one": np.full(M, 17), "runs": np.arange(M) // 50,
               "distinct": rng.permutation(n)[:M],
               "outside": np.where(rng.random(M) < 0.5, rng.choice([-5, n, n + 9, 2 ** 31 - 1], M),
                                   rng.integers(0, n, M))}[ids]
    run(rng, M, 264, 264, 16, n, "bf16", "bf16", ids=pattern)
    run(rng, M, 264, 264, 16, n, "bf16", "f32", ids=pattern, scale=False, order=(1, 1, 0))


@pytest.mark.parametrize("act,bias", [(0, True), (1, True), (2, True), (2, False)])
@pytest.mark.parametrize("M", [9, 300])
def test_lora_epilogue(act, bias, M):
    rng = np.random.default_rng(act)
    run(rng, M, 136, 520, 16, 5, "bf16", "bf16", act=act, bias=bias)
    run(rng, M, 136, 520, 16, 5, "f16", "f32", act=act, bias=bias)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_lora_large(dtype):
    rng = np.random.default_rng(31)
    M = 1500
    ids = np.sort(rng.integers(-1, 6, M))
    run(rng, M, 512, 4096, 64, 6, dtype, dtype, ids=ids)
    run(rng, M, 512, 2048, 16, 6, dtype, "f32", ids=ids, order=(0, 0, 0))


def test_lora_unaligned_operands():
    rng = np.random.default_rng(32)
    run(rng, 70, 77, 51, 5, 4, "bf16", "f32", pad=1)
    run(rng, 70, 77, 51, 5, 4, "f16", "f16", order=(0, 0, 0), pad=1)


def test_lora_without_adapters_is_the_projection():
    rng = np.random.default_rng(33)
    for n, rank in ((0, 16), (3, 0)):
        run(rng, 20, 72, 80, rank, n, "bf16", "f32", ids=np.zeros(20))


@pytest.mark.parametrize("M", [6, 200])
@pytest.mark.parametrize("bad", ["LA", "LB"])
def test_lora_special_values_stay_with_their_adapter(M, bad):
    # one adapter full of NaNs and infinities: rows of the other adapters do not change
    rng = np.random.default_rng(34)
    X, W, LA, LB = operands(rng, M, 264, 300, 16, 4, "bf16", (1, 1, 1))
    t = LA if bad == "LA" else LB
    t[2] = float("nan")
    t[2, 0] = float("inf")
    ids = torch.from_numpy((np.arange(M) % 5 - 1).astype(np.int32)).cuda()
    got = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
    done()
    t[2] = 0.0
    ref, tol = lora_ref(X, W, LA, LB, ids, None, None, 0, "bf16", "f32")
    ok = ids.cpu().numpy() != 2
    assert_close(got[torch.from_numpy(ok).cuda()], ref[ok], tol[ok], "f32")
    assert not bool(torch.isfinite(got[torch.from_numpy(~ok).cuda()]).any())


def test_lora_gradients_match_the_formula_and_differences():
    """dX is the same call with the factors exchanged; the adapters' gradients
    are the grouped weight gradients of the rows grouped by adapter."""
    rng = np.random.default_rng(35)
    M, K, N, r, n = 150, 72, 88, 16, 4
    X, W, LA, LB = operands(rng, M, K, N, r, n, "bf16", (1, 1, 1))
    ids = torch.from_numpy(rng.integers(-1, n, M).astype(np.int32)).cuda()
    s = torch.from_numpy((rng.random(n) + 0.5).astype(np.float32)).cuda()
    G = padded(draw(rng, (M, N), "bf16"), 8)
    dX = lib.gemm_lora(G, W.t(), LB.transpose(1, 2), LA.transpose(1, 2), ids, scale=s,
                       out_dtype=torch.float32)
    done()
    ref, tol = lora_ref(G, W.t(), LB.transpose(1, 2), LA.transpose(1, 2), ids, s, None, 0, "bf16",
                        "f32")
    assert_close(dX, ref, tol, "f32")
    # directional difference of L = sum(G D), linear in X (steps that BF16 holds exactly)
    E = torch.from_numpy(rng.integers(-1, 2, (M, K)).astype(np.float32)).cuda()
    Xi = torch.from_numpy(rng.integers(-3, 4, (M, K)).astype(np.float32)).cuda()

    def loss(x):
        D = lib.gemm_lora(x.to(torch.bfloat16), W, LA, LB, ids, scale=s, out_dtype=torch.float32)
        return float((D.double() * G.double()).sum())

    quotient = (loss(Xi + E) - loss(Xi - E)) / 2
    _, t = lora_ref((Xi.abs() + E.abs()).to(torch.bfloat16), W, LA, LB, ids, s, None, 0, "bf16", "f32")
    size = float((np.abs(G.double().cpu().numpy()) * t).sum())
    want = float((dX.double() * E.double()).sum())
    slack = float((np.abs(E.double().cpu().numpy()) * tol).sum())
    assert abs(quotient - want) <= 2 * size + 2 * slack
    # adapter gradients: rows in adapter order, U = s X LA, V = s G LB^T
    offsets, order, _ = lib.group_rows(ids, n)
    rows = order[:int(offsets[-1])].long()
    mine = ids[rows].long()
    u = torch.einsum("mk,mkr->mr", X[rows].float(), LA.float()[mine]) * s[mine][:, None]
    dLB = lib.gemm_grouped_wgrad(u.to(torch.bfloat16), G[rows].contiguous(), offsets)
    done()
    ref, tol = wgrad_ref(u.to(torch.bfloat16), G[rows], offsets.cpu().numpy(), None, None, 1.0, 0.0)
    assert_close(dLB, ref, tol, "f32")


def test_lora_streams_graphs_and_repeats():
    rng = np.random.default_rng(36)
    M = 90
    X, W, LA, LB = operands(rng, M, 264, 392, 16, 8, "bf16", (1, 1, 1))
    ids = torch.from_numpy(rng.integers(-1, 8, M).astype(np.int32)).cuda()
    first = lib.gemm_lora(X, W, LA, LB, ids)
    done()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = lib.gemm_lora(X, W, LA, LB, ids)
    side.synchronize()
    assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.gemm_lora(X, W, LA, LB, ids)
    ids.copy_(torch.from_numpy(rng.integers(-1, 8, M).astype(np.int32)))
    graph.replay()
    done()
    ref, tol = lora_ref(X, W, LA, LB, ids, None, None, 0, "bf16", "bf16")
    assert_close(out, ref, tol, "bf16")


def test_lora_many_slots_in_several_launches():
    # 128 slots of 2 x 256 columns per tile: V of 1100 rows passes its 128 MiB
    rng = np.random.default_rng(37)
    run(rng, 1100, 72, 136, 256, 300, "bf16", "f32")
    run(rng, 9, 72, 136, 300, 4, "f16", "f16")  # a rank past the tensor-core path's


def test_lora_one_adapter_for_all_numbers():
    # stacks of stride 0: every number names the same matrices
    rng = np.random.default_rng(38)
    for M in (20, 300):
        X, W, LA, LB = operands(rng, M, 136, 264, 16, 1, "bf16", (1, 1, 1))
        LA, LB = LA.expand(5, 136, 16), LB.expand(5, 16, 264)
        ids = torch.from_numpy(rng.integers(-1, 5, M).astype(np.int32)).cuda()
        got = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
        done()
        ref, tol = lora_ref(X, W, LA, LB, ids, None, None, 0, "bf16", "f32")
        assert_close(got, ref, tol, "f32")
