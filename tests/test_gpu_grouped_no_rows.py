"""Products whose rows are all gathered from an A without rows: rows of zeros."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import done

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_rows_of_an_empty_a(dtype):
    offsets = torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")
    index = torch.tensor([-1, 0, 3, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    A = torch.empty((0, 16), dtype=dtype, device="cuda")
    B = torch.ones((3, 16, 24), dtype=dtype, device="cuda")
    bias = torch.arange(3 * 24, dtype=torch.float32, device="cuda").reshape(3, 24)
    D = lib.gemm_grouped(A, B, offsets, row_index=index, bias=bias, out_dtype=torch.float32)
    C = bias.view(3, 1, 24).expand(3, 16, 24).contiguous()
    G = lib.gemm_grouped_wgrad(A, torch.ones((5, 24), dtype=dtype, device="cuda"), offsets,
                               row_index=index, C=C, beta=0.5)
    done()
    assert torch.equal(D, bias[[0, 0, 2, 2, 2]])
    assert torch.equal(G, 0.5 * C)
