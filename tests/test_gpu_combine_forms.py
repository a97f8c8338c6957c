"""Forms of combine_grad beside the ones that the helper makes of whole, aligned batches: the weights'
gradient alone, and dD off 16 bytes in large batches."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH

pytestmark = pytest.mark.gpu
TYPE = {"f32": lib.GEMM_D_F32, "bf16": lib.GEMM_D_BF16, "f16": lib.GEMM_D_F16}


@pytest.mark.parametrize("y,d", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32")])
@pytest.mark.parametrize("T,k,N,bulk", [(7, 3, 100, False), (300, 8, 1031, False), (2048, 2, 2048, True),
                                        (1701, 2, 9001, True), (1777, 8, 2100, True), (1640, 11, 2056, True)])
def test_the_weights_gradient_alone(y, d, T, k, N, bulk):
    """dY == NULL: dweights has the same bits as with it."""
    ld = -(-N // 8) * 8
    g = torch.Generator(device="cuda").manual_seed(T)
    Y = torch.empty(T * k, ld, dtype=TORCH[y], device="cuda").normal_(generator=g)
    dD = torch.empty(T, ld, dtype=TORCH[d], device="cuda").normal_(generator=g)
    at = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    at[::3, 0] = -1
    dY = torch.empty_like(Y)
    both, alone = (torch.full((T, k), float("nan"), device="cuda") for _ in range(2))
    args = (T, k, N, dD, ld, TYPE[d], Y, ld, T * k, TYPE[y], at, None)
    for rows, dw in ((dY, both), (None, alone)):
        lib.gemm_combine_grad(*args, rows, ld, dw)
        assert lib.gemm_last_kernel() == ("combine_grad<bulk>" if bulk else "combine_grad")
    rows = Y.double()[at.long().clamp(min=0), :N] * (at >= 0)[..., None]
    ref = (dD[:, None, :N].double() * rows).sum(-1)
    # (a thread's share: at most N / 32 products and 8, then 5 shuffles and 8 warps)
    tol = (dD[:, None, :N].double().abs() * rows.abs()).sum(-1) * (N / 32 + 24) * 2.0 ** -24
    assert ((alone.double() - ref).abs() <= tol).all()
    assert torch.equal(alone, both)
    assert lib.gemm_last_device_status() == lib.GEMM_OK


@pytest.mark.parametrize("y,d", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                 ("f16", "f32")])
@pytest.mark.parametrize("T,k,N", [(4100, 1, 8192), (1701, 2, 9001), (1777, 8, 2100), (1640, 11, 2055),
                                   (4500, 2, 1032)])
def test_large_batches_with_dd_off_16_bytes(y, d, T, k, N):
    """dD's rows come by ordinary loads, Y's by bulk copy: the same bits as with dD on 16 bytes."""
    ld = -(-N // 8) * 8
    g = torch.Generator(device="cuda").manual_seed(N)
    Y = torch.empty(T * k, ld, dtype=TORCH[y], device="cuda").normal_(generator=g)[:, :N]
    dD = torch.empty(T, ld, dtype=TORCH[d], device="cuda").normal_(generator=g)[:, :N]
    odd = torch.full((T, N + 1), float("nan"), dtype=TORCH[d], device="cuda")[:, 1:]
    odd.copy_(dD)
    at = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    at[::4, 0] = -1
    w = torch.rand(T, k, generator=g, device="cuda")
    store = [torch.zeros(T * k, ld, dtype=TORCH[y], device="cuda")[:, :N] for _ in range(2)]
    want, dw = lib.combine_grad(dD, Y, at, weights=w, out=store[0])
    name = lib.gemm_last_kernel()
    got, ow = lib.combine_grad(odd, Y, at, weights=w, out=store[1])
    assert lib.gemm_last_kernel() == name
    row = N * Y.element_size()
    bulk = row >= 1280 and row * k >= 4096 and row * k * T >= (64 if k == 1 else 16) << 20
    assert name == ("combine_grad<bulk>" if bulk else "combine_grad")
    assert torch.equal(got, want) and torch.equal(ow, dw)
    assert lib.gemm_last_device_status() == lib.GEMM_OK
