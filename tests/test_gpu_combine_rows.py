"""combine_grad's rows that no token has: 0 in a new tensor, left alone in a given one."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH

pytestmark = pytest.mark.gpu


def poison(rows, N, dtype, stream=None):
    """Memory of NaNs for the allocator to hand out again."""
    with torch.cuda.stream(stream):
        for _ in range(4):
            t = torch.full((rows, N), float("nan"), dtype=dtype, device="cuda")
            del t


def batch(T, k, N, rows, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Y = torch.randn(rows, N, device="cuda", generator=g).to(dtype)
    at = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)  # (past the last row: none)
    at[::5] = -1
    at = at.view(T, k)
    w = torch.rand(T, k, generator=g, device="cuda")
    dD = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    named = torch.zeros(rows, dtype=torch.bool, device="cuda")
    named[at[(at >= 0) & (at < rows)].long()] = True
    return Y, at, w, dD, named


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,N,rows", [(1, 1, 1, 3), (5, 3, 40, 15), (40, 4, 257, 130), (40, 4, 256, 400),
                                        (3400, 2, 2048, 6000)])
def test_new_rows_without_a_token_are_zero(dtype, T, k, N, rows):
    """A gradient of what adds nothing is 0, and no memory that something else has left."""
    Y, at, w, dD, named = batch(T, k, N, rows, TORCH[dtype])
    side = torch.cuda.Stream()
    kept = torch.full((rows, N), 7.0, dtype=TORCH[dtype], device="cuda")
    lib.combine_grad(dD, Y, at, weights=w, out=kept)
    assert (kept[~named] == 7.0).all()  # (rows of a given tensor stay)
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        poison(rows, N, TORCH[dtype], None if stream is None else side)
        torch.cuda.synchronize()
        for weights in (True, False):
            dY, _ = lib.combine_grad(dD, Y, at, weights=w, weight_grad=weights, stream=stream)
            torch.cuda.synchronize()
            assert (dY[~named] == 0).all()
            assert torch.equal(dY[named], kept[named])
            dY.fill_(float("nan"))
            torch.cuda.synchronize()
            del dY


def test_no_choices_and_no_rows():
    Y, at, w, dD, _ = batch(20, 2, 64, 40, torch.bfloat16)
    poison(40, 64, torch.bfloat16)
    dY, dw = lib.combine_grad(dD, Y, at[:, :0].contiguous())
    assert (dY == 0).all() and dw.shape == (20, 0)
    dY, dw = lib.combine_grad(dD[:0], Y, at[:0], weights=w[:0])
    assert (dY == 0).all() and dY.shape == Y.shape


def test_new_rows_in_a_graph():
    """Each replay leaves 0 in the rows that its positions do not name."""
    Y, at, w, dD, named = batch(64, 4, 512, 256, torch.float16)
    want, _ = lib.combine_grad(dD, Y, at, weights=w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dY, _ = lib.combine_grad(dD, Y, at, weights=w)
    for _ in range(2):
        dY.fill_(float("nan"))
        graph.replay()
        assert torch.equal(dY, want)
    at.fill_(-1)
    graph.replay()
    assert (dY == 0).all()
