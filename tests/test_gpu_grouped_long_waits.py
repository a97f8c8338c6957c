"""Sums so long that one tile takes more than a second: the waits' limit grows
with them, and the result is complete.

The partial sums stay small (ones against ones of alternating sign, 64 at a time,
the first block twice), so every addition is exact and the sum is 64."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import done

pytestmark = pytest.mark.gpu


def alternating(steps, columns, dtype):
    t = torch.ones((steps, columns), dtype=dtype, device="cuda")
    t.view(-1, 2, 64, columns)[:, 1] = -1
    t[:64] = 2
    return t


def test_a_product_of_two_thousand_million_steps():
    K, N = (1 << 31) - 128, 8
    A = torch.ones((1, K), dtype=torch.bfloat16, device="cuda")
    B = torch.empty((1, N, K), dtype=torch.bfloat16, device="cuda")
    B[0] = alternating(K, 1, torch.bfloat16).view(1, K)
    offsets = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    D = lib.gemm_grouped(A, B.transpose(1, 2), offsets)
    end.record()
    done()
    print(f"{start.elapsed_time(end):.0f} ms")
    assert bool((D == 64).all())


def test_a_weight_gradient_of_five_hundred_million_rows():
    rows, M, N = 1 << 29, 8, 8
    A = torch.ones((rows, M), dtype=torch.bfloat16, device="cuda")
    B = alternating(rows, N, torch.bfloat16)
    offsets = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    D = lib.gemm_grouped_wgrad(A, B, offsets, out_dtype=torch.bfloat16)
    end.record()
    done()
    print(f"{start.elapsed_time(end):.0f} ms")
    assert bool((D == 64).all())
