"""FP32 weight gradients of groups of very different length: a long group's sums
are as good as if it were alone, however many short or empty groups share the
call.  Tolerance as for long sums (test_gpu_long_sums.py)."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import done, offsets_of
from test_gpu_long_sums import long_tolerance, normal, off_by

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes", [[3] * 60 + [16000] + [5] * 68, [0] * 500 + [14000, 0, 0, 1],
                                   [1000, 0, 0, 0, 0, 0, 0], [769] + [0] * 700])
@pytest.mark.parametrize("M,N,beta", [(128, 256, 0.0), (264, 500, 1.0)])
def test_one_long_group_among_short_ones(dtype, sizes, M, N, beta):
    rows, groups = sum(sizes), len(sizes)
    long = int(np.argmax(sizes))
    A, B = normal(21, (rows, M), dtype), normal(22, (rows, -(-N // 8) * 8), dtype)[:, :N]
    C = normal(23, (1, M, N), "f32").expand(groups, M, N) if beta else None
    off = offsets_of(sizes)
    D = lib.gemm_grouped_wgrad(A, B, torch.from_numpy(off).cuda(), C=C, beta=beta)
    name = lib.gemm_last_kernel()
    done()
    assert name.startswith("wgrad_tc")
    for g in (long, (long + 1) % groups):
        lo, hi = int(off[g]), int(off[g + 1])
        ref = A[lo:hi].double().t() @ B[lo:hi].double()
        if beta:
            ref += C[g].double()
        if hi > lo or beta:
            assert off_by(D[g], ref) <= long_tolerance(max(hi - lo, 1)), (name, g)
        else:
            assert not bool(D[g].any())
