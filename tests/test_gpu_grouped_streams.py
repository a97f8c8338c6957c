"""The grouped helpers on a stream of the caller's: their outputs are memory that
no work of the current stream still uses."""
import pytest
import torch

import dense_gemm_08_gb300 as lib

pytestmark = pytest.mark.gpu

ROWS, K, N, GROUPS = 96, 64, 128, 3


def inputs():
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)

    A, B, G = normal(ROWS, K), normal(GROUPS, K, N), normal(ROWS, N)
    W, LA, LB = normal(K, N), normal(GROUPS, K, 8), normal(GROUPS, 8, N)
    off = torch.tensor([0, 30, 31, ROWS], dtype=torch.int32, device="cuda")
    ids = (torch.arange(ROWS, device="cuda") % GROUPS).to(torch.int32)
    return {
        "gemm_grouped": lambda s: lib.gemm_grouped(A, B, off, stream=s),
        "gemm_grouped_wgrad": lambda s: lib.gemm_grouped_wgrad(A, G, off, stream=s),
        "gemm_lora": lambda s: lib.gemm_lora(A, W, LA, LB, ids, stream=s),
        "group_rows": lambda s: lib.group_rows(ids, GROUPS, stream=s)[1],
    }


@pytest.mark.parametrize("name", ["gemm_grouped", "gemm_grouped_wgrad", "gemm_lora", "group_rows"])
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_belong_to_the_stream(name, handle):
    call = inputs()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    # a freed tensor of the output's size that the current stream has yet to write
    stale = torch.empty_like(want)
    at = stale.data_ptr()
    torch.cuda._sleep(200_000_000)
    stale.fill_(7)
    del stale
    got = call(side.cuda_stream if handle else side)
    assert got.data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["gemm_grouped", "gemm_grouped_wgrad", "gemm_lora", "group_rows"])
def test_the_default_stream_by_its_handle(name):
    call = inputs()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = call(0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
