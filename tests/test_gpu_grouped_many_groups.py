"""Row products over millions of groups, nearly all of them empty."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import done

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups", [1 << 20, 1 << 24])
def test_rows_in_the_first_and_the_last_groups(dtype, groups):
    rows, K, N = 200, 64, 72
    g = torch.Generator(device="cuda").manual_seed(2)
    A = torch.empty((rows, K), dtype=dtype, device="cuda").normal_(generator=g)
    B = torch.empty((1, K, N), dtype=dtype, device="cuda").normal_(generator=g)
    offsets = torch.full((groups + 1,), 70, dtype=torch.int32, device="cuda")
    offsets[0], offsets[-2], offsets[-1] = 0, 130, rows
    D = lib.gemm_grouped(A, B.expand(groups, K, N), offsets, out_dtype=torch.float32)
    done()
    ref = A.double() @ B[0].double()
    assert float((D.double() - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
