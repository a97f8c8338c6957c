"""A NaN of a row reaches that row's results, whatever the activation."""
import itertools

import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import (TORCH, assert_close, done, draw, grouped_ref, lora_ref, offsets_of,
                             padded)

pytestmark = pytest.mark.gpu

ACTS = [lib.GEMM_ACT_NONE, lib.GEMM_ACT_RELU, lib.GEMM_ACT_GELU]


def check(D, ref, tol, out, row):
    keep = np.arange(ref.shape[0]) != row
    at = torch.from_numpy(keep).cuda()
    assert bool(torch.isnan(D[~at]).all())
    assert_close(D[at], ref[keep], tol[keep], out)


# pad 1: rows of 77 and 51 values, which the CUDA cores take; 200 columns: stores in quads
@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                       ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("act,pad", list(itertools.product(ACTS, [1, 8])))
@pytest.mark.parametrize("K", [77, 1000])
def test_grouped(dtype, out, act, pad, K):
    rng = np.random.default_rng(act + pad)
    sizes, N = [40, 0, 3], 51 if pad == 1 else 200
    A = padded(draw(rng, (43, K), dtype), pad)
    A[17, 5] = float("nan")
    B = padded(draw(rng, (3, K, N), dtype, sigma=K ** -0.5), pad)
    off = offsets_of(sizes)
    D = lib.gemm_grouped(A, B, torch.from_numpy(off).cuda(), activation=act, out_dtype=TORCH[out])
    done()
    A = A.clone()
    A[17, 5] = 0
    ref, tol, _ = grouped_ref(A, B, off, None, None, act, 1.0)
    check(D, ref, tol, out, 17)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("act,pad", list(itertools.product(ACTS, [1, 8])))
@pytest.mark.parametrize("M", [9, 150])
def test_lora(dtype, out, act, pad, M):
    rng = np.random.default_rng(act + pad)
    K, N, n, r = 77, 51, 3, 8
    X = padded(draw(rng, (M, K), dtype), pad)
    W = padded(draw(rng, (K, N), dtype, sigma=0.1), pad)
    LA = padded(draw(rng, (n, K, r), dtype, sigma=0.1), pad)
    LB = padded(draw(rng, (n, r, N), dtype, sigma=0.5), pad)
    ids = torch.from_numpy((np.arange(M) % (n + 1) - 1).astype(np.int32)).cuda()
    X[6, 70] = float("nan")
    D = lib.gemm_lora(X, W, LA, LB, ids, activation=act, out_dtype=TORCH[out])
    done()
    X = X.clone()
    X[6, 70] = 0
    ref, tol = lora_ref(X, W, LA, LB, ids, None, None, act, dtype, out)
    check(D, ref, tol, out, 6)
