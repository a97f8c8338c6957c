"""dbias where a long K is split over a cluster: as exact as where a CTA sums all of it, in parts of 768."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH

pytestmark = pytest.mark.gpu

# An addition of sixteen products to the accumulator cuts its last place: half a unit on the mean, that is
# between 2^-25 and 2^-24 of the sum so far.  With operands of one sign the sum grows evenly, so that a part of 768,
# 48 additions, loses at most 24.5 * 2^-24 = 1.46e-6 of itself (a piece of 1024 1.94e-6, of 2048 3.9e-6;
# measured 1.74e-6 for 1024).  What else is rounded -- D's sum of parts and pieces, the columns' sums -- is rounded to
# nearest, either way: a tenth of that in a column's mean.
MOST = 1.46e-6 + 0.15e-6


def one_sign(M, N, K, dtype, ob, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    A = torch.empty(M, K, device="cuda").normal_(generator=g).abs_() + 0.1
    B = (torch.empty(K, N, device="cuda").normal_(generator=g).abs_() + 0.1) * K ** -0.5
    A, B = A.to(TORCH[dtype]), B.to(TORCH[dtype])
    return A, (B.t().contiguous().t() if ob else B)


def loss(M, N, K, dtype, ob):
    """(mean relative error of dbias, kernel)"""
    A, B = one_sign(M, N, K, dtype, ob)
    D, sums = lib.gemm_fused_grad(A, B, None, bias_grad=True)
    name = lib.gemm_last_kernel()
    ref = (A.double() @ B.double())
    size = ref.sum(0)
    # (every term is positive: a part that is left out or added twice is off by far more)
    assert ((sums.double() - size).abs() <= 2e-5 * size).all()
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    assert ((D.double() - ref).abs() <= ref * (step + 2e-5)).all()
    again, sums2 = lib.gemm_fused_grad(A, B, None, bias_grad=True)
    assert torch.equal(again, D) and torch.equal(sums2, sums)
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    return float((sums.double() - size).sum() / size.sum()), name


# (None: whichever way the library takes)
CUTS = [("split", 64, 1000, 8192), ("split", 16, 200, 8192), ("split", 33, 64, 8000), ("split", 64, 64, 4096),
        ("split", 256, 256, 6000), (None, 64, 1000, 12288), (None, 100, 520, 16384), (None, 256, 512, 24576),
        (None, 16, 72, 40000), (None, 128, 2048, 10000), (None, 8, 8, 6152), (None, 500, 1032, 4104)]


@pytest.mark.parametrize("ob", [0, 1])
@pytest.mark.parametrize("way,M,N,K", CUTS)
def test_bf16_sums_of_one_sign(ob, way, M, N, K):
    off, name = loss(M, N, K, "bf16", ob)
    assert way is None or way in name
    assert abs(off) <= MOST, name


@pytest.mark.parametrize("ob", [0, 1])
@pytest.mark.parametrize("way,M,N,K", CUTS)
def test_f16_sums_as_of_one_cta(ob, way, M, N, K):
    """(Products of FP16 are longer than an accumulator's last place: they are cut as well, some four times as
    much in all.  The measure is a product of many tiles, each summed by one CTA pair in parts of 768.)"""
    whole, name = loss(2304, 2560, 2304, "f16", ob)
    assert "pair" in name
    off, name = loss(M, N, K, "f16", ob)
    assert way is None or way in name
    assert abs(off) <= 1.1 * abs(whole) + 0.15e-6, name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(64, 1000, 8192), (16, 200, 8192), (33, 64, 8000), (300, 130, 9000)])
def test_sums_in_graphs_and_on_streams(dtype, M, N, K):
    A, B = one_sign(M, N, K, dtype, 0)
    Z = torch.randn(M, N, device="cuda").to(A.dtype)
    want, sums = lib.gemm_fused_grad(A, B, Z, activation=lib.GEMM_ACT_GELU, bias_grad=True)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(4)]
    got = [lib.gemm_fused_grad(A, B, Z, activation=lib.GEMM_ACT_GELU, bias_grad=True, stream=s) for s in sides * 4]
    torch.cuda.synchronize()
    assert all(torch.equal(d, want) and torch.equal(s, sums) for d, s in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d, s = lib.gemm_fused_grad(A, B, Z, activation=lib.GEMM_ACT_GELU, bias_grad=True)
    for _ in range(3):
        d.zero_(), s.zero_()
        graph.replay()
        assert torch.equal(d, want) and torch.equal(s, sums)
    assert lib.gemm_last_device_status() == lib.GEMM_OK
