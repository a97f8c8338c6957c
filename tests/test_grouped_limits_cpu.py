"""Sizes past what the grouped operators' kernels count are refused before any
CUDA call."""
import pytest

import dense_gemm_08_gb300 as lib

FAKE = 1 << 20  # never dereferenced: the checks run before any CUDA call


@pytest.mark.parametrize("fn_name", ["gemm_grouped_f32", "gemm_grouped_bf16_f32acc",
                                     "gemm_grouped_f16_f32acc"])
@pytest.mark.parametrize("groups", [(1 << 24) + 1, (1 << 31) - 32, (1 << 31) - 1])
def test_more_groups_than_a_walk_takes(fn_name, groups):
    a = dict(groups=groups, rows=9, N=16, K=8, alpha=1.0, A=FAKE, lda=8, rows_a=9, row_index=None,
             offsets=FAKE, B=FAKE, ldb=16, stride_b=0, order_b=0, D=FAKE, ldd=16)
    assert getattr(lib, fn_name)(**a, stream=0, check=False) == lib.GEMM_ERR_INVALID_VALUE
