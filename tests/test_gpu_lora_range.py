"""gemm_lora in FP16 where the first product leaves FP16's range: the result is
the definition's, which may lie well inside it."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH, assert_close, done, lora_ref, rel_sum
from test_gpu_lora import operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 7, 90, 300])
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("order", [(1, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("rank", [16, 40])
def test_first_product_past_the_largest_value(M, out, order, rank):
    # rows of one adapter in three have X LA of some 2^17, their LB is small
    rng = np.random.default_rng(M + rank)
    K, N, n = 264, 200, 3
    X, W, LA, LB = operands(rng, M, K, N, rank, n, "f16", order)
    LA[1] *= 2.0 ** 13
    LB[1] *= 2.0 ** -13
    X *= 16
    ids = torch.from_numpy(((np.arange(M) + 1) % (n + 1) - 1).astype(np.int32)).cuda()
    if M == 1:
        ids[0] = 1
    s = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    first = float((X.double() @ LA[1].double()).abs().max()) * 2
    assert first > 65504
    D = lib.gemm_lora(X, W, LA, LB, ids, scale=s, out_dtype=TORCH[out])
    done()
    ref, tol = lora_ref(X, W, LA, LB, ids, s, None, 0, "f16", out)
    # the K products of a sum computed again are added one by one: K roundings of 2^-24
    x, w = np.abs(X.double().cpu().numpy()), np.abs(W.double().cpu().numpy())
    tol = tol + K * 2.0 ** -24 * (x @ w)
    assert rel_sum(K) < 1e-3 and np.isfinite(ref).all()
    assert_close(D, ref, tol, out)


def test_past_it_beside_another_adapters_infinities():
    rng = np.random.default_rng(5)
    M, K, N = 40, 264, 200
    X, W, LA, LB = operands(rng, M, K, N, 16, 3, "f16", (1, 1, 1))
    LA[1] *= 2.0 ** 13
    LB[1] *= 2.0 ** -13
    X *= 16
    ids = torch.from_numpy((np.arange(M) % 4 - 1).astype(np.int32)).cuda()
    dirty = LB.clone()
    dirty[2, 3, 7], dirty[2, 4, 8], dirty[0, 1, 9] = float("inf"), float("nan"), float("-inf")
    D = lib.gemm_lora(X, W, LA, dirty, ids, out_dtype=torch.float32)
    done()
    ref, tol = lora_ref(X, W, LA, LB, ids, None, None, 0, "f16", "f32")
    x, w = np.abs(X.double().cpu().numpy()), np.abs(W.double().cpu().numpy())
    tol = tol + K * 2.0 ** -24 * (x @ w)
    keep = (ids.cpu().numpy() == 1) | (ids.cpu().numpy() == -1)
    assert_close(D[torch.from_numpy(keep).cuda()], ref[keep], tol[keep], "f32")


@pytest.mark.parametrize("M", [3, 90, 300])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("down", [0, 8, 14, 20, 30])
def test_small_first_products(M, dtype, out, down):
    """The documented bound: 2^-8 (an FP32 D 2^-15) of sum |u LB|, and with FP16 inputs
    2^-25 sum |LB|; u = scale * X LA down to far below FP16's smallest step."""
    out = dtype if out == "same" else out
    rng = np.random.default_rng(M + down)
    K, N, rank, n = 264, 200, 16, 3
    X, W, LA, LB = operands(rng, M, K, N, rank, n, dtype, (1, 1, 1))
    W *= 0  # (the second product alone)
    LB *= 2.0 ** 12
    ids = torch.from_numpy((np.arange(M) % (n + 1) - 1).astype(np.int32)).cuda()
    s = torch.full((n,), 2.0 ** -down, device="cuda")
    D = lib.gemm_lora(X, W, LA, LB, ids, scale=s, out_dtype=TORCH[out])
    done()
    ref, tol = np.zeros((M, N)), np.zeros((M, N))
    x, la, lb = (t.double().cpu().numpy() for t in (X, LA, LB))
    for i, a in enumerate(ids.tolist()):
        if a < 0:
            continue
        u = 2.0 ** -down * (x[i] @ la[a])
        summed = rel_sum(K) * 2.0 ** -down * (np.abs(x[i]) @ np.abs(la[a]))  # u's own sum
        ref[i] = u @ lb[a]
        part = 2.0 ** -15 if out == "f32" else 2.0 ** -8
        tol[i] = (part * np.abs(u) + rel_sum(rank) * np.abs(u) + summed) @ np.abs(lb[a])
        if dtype == "f16":
            tol[i] += 2.0 ** -25 * np.abs(lb[a]).sum(0)
    assert_close(D, ref, tol, out)
