"""FP32 results of long sums of 16-bit products.  The tensor cores cut what an
addition cannot hold, always towards zero, so one accumulator's error grows
with the sum's length (about 2e-5 of the result after 16384 products); the
grouped products and the weight gradients make such sums in parts.

Tolerance, in the 2-norm: a step adds 16 products and may cut two units of the
last of 24 bits (2^-22 of the accumulator); a part has 768 products, 48 steps,
and each of the ceil(K / 768) parts is added with one rounding (2^-24):
48 * 2^-22 + parts * 2^-24, which is below 1.3e-5 up to 16384 products.
"""
import math

import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH, done, offsets_of
from test_gpu_grouped import run_grouped, run_wgrad

pytestmark = pytest.mark.gpu


def long_tolerance(K):
    return 48 * 2.0 ** -22 + math.ceil(K / 768) * 2.0 ** -24


def normal(seed, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=TORCH[dtype], device="cuda").normal_(generator=g)


def off_by(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def on_device(sizes):
    return torch.from_numpy(offsets_of(sizes)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,N,gather", [([9], 200, True), ([40], 264, False), ([200], 1000, True),
                                            ([1024], 19 * 256, False)])
def test_grouped(dtype, sizes, N, gather):
    K, rows = 16384, sum(sizes)
    A, B = normal(1, (rows, K), dtype), normal(2, (len(sizes), N, K), dtype).transpose(1, 2)
    index = None
    if gather:
        index = torch.from_numpy(np.random.default_rng(3).permutation(rows).astype(np.int32)).cuda()
    D = lib.gemm_grouped(A, B, on_device(sizes), row_index=index, out_dtype=torch.float32)
    name = lib.gemm_last_kernel()
    done()
    ref = (A if index is None else A[index.long()]).double() @ B[0].double()
    assert off_by(D, ref) <= long_tolerance(K), name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(128, 256), (100, 251), (2560, 2048), (2560, 2047)])
@pytest.mark.parametrize("beta", [0.0, 1.0])
def test_wgrad(dtype, M, N, beta):
    rows = 16384
    A = normal(4, (rows, -(-M // 8) * 8), dtype)[:, :M]
    B = normal(5, (rows, -(-N // 8) * 8), dtype)[:, :N]
    C = normal(6, (1, M, N), "f32") if beta else None
    D = lib.gemm_grouped_wgrad(A, B, on_device([rows]), C=C, beta=beta)
    name = lib.gemm_last_kernel()
    done()
    ref = A.double().t() @ B.double()
    if beta:
        ref += C[0].double()
    assert off_by(D[0], ref) <= long_tolerance(rows), name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [767, 768, 769, 1536, 1544])
@pytest.mark.parametrize("order", [0, 1])
def test_grouped_ends_of_parts(dtype, K, order):
    rng = np.random.default_rng(K)
    run_grouped(rng, [3, 0, 70, 129], 2, K, 77, dtype, order, "f32", bias=True, act=lib.GEMM_ACT_GELU,
                alpha=-0.5)
    run_grouped(rng, [5, 0, 2], 1, K, 96, dtype, order, "f32", gather=True, bias=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,pad_d", [(96, 0), (77, 0), (96, 1)])
@pytest.mark.parametrize("alpha,beta,in_place", [(1.0, 0.0, False), (0.5, 0.0, False),
                                                 (1.0, 1.0, True), (-2.0, 0.25, False)])
def test_wgrad_ends_of_parts(dtype, N, pad_d, alpha, beta, in_place):
    rng = np.random.default_rng(N + pad_d)
    for sizes in ([767, 768, 769], [0, 1537, 1, 2305, 0], [4000]):
        run_wgrad(rng, sizes, 3, 72, N, dtype, "f32", alpha=alpha, beta=beta, in_place=in_place,
                  pad_d=pad_d, gather=sizes[0] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_integer_sums_are_exact(dtype):
    rng = np.random.default_rng(7)
    run_grouped(rng, [130, 0, 60], 0, 4000, 100, dtype, 1, "f32", dist="int")
    run_wgrad(rng, [2000, 0, 900], 0, 130, 100, dtype, "f32", dist="int")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_special_values_in_long_sums(dtype):
    """Infinities and NaNs of one group stay in it, whichever part they are in."""
    sizes, M, N = [1000, 900, 1100], 64, 96
    A, B = normal(8, (sum(sizes), M), dtype), normal(9, (sum(sizes), N), dtype)
    clean = lib.gemm_grouped_wgrad(A, B, on_device(sizes))
    A[1000 + 20, 3] = float("inf")
    B[1000 + 850, 5] = float("nan")
    D = lib.gemm_grouped_wgrad(A, B, on_device(sizes))
    done()
    assert torch.equal(D[0], clean[0]) and torch.equal(D[2], clean[2])
    assert not bool(torch.isfinite(D[1, 3]).any())
    assert bool(torch.isnan(D[1, :, 5]).all())


def adapters(seed, dtype, n, K, N, rank):
    return (normal(seed, (n, rank, K), dtype).transpose(1, 2),
            (normal(seed + 1, (n, N, rank), dtype) * 0.01).transpose(1, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 512), (40, 200), (200, 999), (600, 26 * 256)])
def test_lora(dtype, M, N):
    """The adapters' part is a hundredth of the result, so its rounding (2^-15 at
    most) is below the tolerance's last digit."""
    K, n, rank = 16384, 5, 16
    X, W = normal(10, (M, K), dtype), normal(11, (N, K), dtype).t()
    LA, LB = adapters(12, dtype, n, K, N, rank)
    ids = torch.from_numpy(np.random.default_rng(14).integers(-1, n, M).astype(np.int32)).cuda()
    scale = torch.full((n,), 0.25, device="cuda")
    D = lib.gemm_lora(X, W, LA, LB, ids, scale=scale, out_dtype=torch.float32)
    name = lib.gemm_last_kernel()
    done()
    ref = X.double() @ W.double()
    for a in range(n):
        rows = ids == a
        ref[rows] += 0.25 * (X[rows].double() @ LA[a].double()) @ LB[a].double()
    assert name.startswith("lora_tc")
    assert off_by(D, ref) <= long_tolerance(K), name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(1, 100), (33, 77), (300, 264), (2000, 2560)])
def test_lora_values_of_other_adapters(dtype, M, N):
    """Infinities and NaNs in one adapter's matrices leave the other rows alone."""
    K, n = 1600, 4
    X, W = normal(15, (M, K), dtype), normal(16, (N, K), dtype).t()
    LA, LB = adapters(17, dtype, n, K, N, 16)
    ids = torch.from_numpy((np.arange(M) % n).astype(np.int32)).cuda()
    clean = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
    LB[2, 3, 5], LB[2, 4, N - 1] = float("inf"), float("nan")
    D = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
    done()
    others = ids != 2
    d, c = D[others].double(), clean[others].double()
    assert bool(torch.isfinite(d).all())
    # recomputed sums are sequential: K roundings of 2^-24 of the absolute sum at most
    S = X[others].double().abs() @ W.double().abs()
    assert bool(((d - c).abs() <= (2 * K * 2.0 ** -24 + long_tolerance(K)) * (S + c.abs() + 1)).all())
    if bool((~others).any()):
        assert not bool(torch.isfinite(D[~others][:, 5]).any())
