"""What gemm_lora takes from the library's pool: X LA of at most 128 MiB at a
time, on the CUDA cores (a rank above 256) as on the tensor cores."""
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import assert_close, done, lora_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_of_a_large_rank(dtype):
    M, K, N, rank, n = 200_000, 8, 16, 512, 3  # X LA in one piece: 390 MiB
    t = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(4)

    def normal(*shape, sigma=1.0):
        return torch.empty(shape, dtype=t, device="cuda").normal_(0, sigma, generator=g)

    X, W = normal(M, K), normal(K, N)
    LA, LB = normal(n, K, rank, sigma=0.3), normal(n, rank, N, sigma=0.05)
    ids = torch.randint(-1, n, (M,), generator=g, device="cuda", dtype=torch.int32)
    torch.cuda.synchronize()
    lib.gemm_release_memory()
    D = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
    held = lib.gemm_memory_info()["pool_reserved_bytes"]
    assert lib.gemm_last_kernel().startswith("lora_simt")
    done()
    assert held <= 160 << 20, held
    for lo in (0, 65530, 131060, M - 30):  # around the launches' ends
        rows = slice(lo, lo + 30)
        ref, tol = lora_ref(X[rows], W, LA, LB, ids[rows], None, None, 0, dtype, "f32")
        assert_close(D[rows], ref, tol, "f32")
    # every row: the last launch's rows are no copies of the first's
    u = torch.einsum("mk,mkr->mr", X[-3000:].float(), LA.float()[ids[-3000:].clamp(min=0).long()])
    v = torch.einsum("mr,mrn->mn", u, LB.float()[ids[-3000:].clamp(min=0).long()])
    want = X[-3000:].float() @ W.float() + v * (ids[-3000:] >= 0)[:, None]
    assert float((D[-3000:] - want).abs().max()) <= 1e-3 * float(want.abs().max())
