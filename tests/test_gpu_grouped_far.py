"""Operands whose rows and matrices lie more than 2^31 elements (and 2^32 bytes)
apart: every offset is counted in 64 bits.  And first calls inside a capture."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import (TORCH, assert_close, done, draw, grouped_ref, lora_ref, offsets_of,
                             wgrad_ref)

pytestmark = pytest.mark.gpu

FAR = (1 << 30) + 8  # elements between rows or matrices; four of them pass 2^32


def far(t, dim):
    """The same values with FAR elements between neighbours of dimension `dim` (the others
    packed); the memory between them is not touched."""
    shape = list(t.shape)
    rest = [n for i, n in enumerate(shape) if i != dim]
    strides, step = [0] * len(shape), 1
    for i in reversed([i for i in range(len(shape)) if i != dim]):
        strides[i] = step
        step *= shape[i] if i != len(shape) - 1 else -(-shape[i] // 8) * 8
    strides[dim] = FAR
    buf = torch.empty(FAR * (shape[dim] - 1) + max(step, 8), dtype=t.dtype, device="cuda")
    assert rest
    out = buf.as_strided(shape, strides)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_grouped_product(dtype):
    rng = np.random.default_rng(1)
    sizes, K, N = [2, 0, 1, 2], 72, 80
    off = offsets_of(sizes)
    at = torch.from_numpy(off).cuda()
    A, B = draw(rng, (5, K), dtype), draw(rng, (4, K, N), dtype, sigma=0.1)
    ref, tol, _ = grouped_ref(A, B, off, None, None, 0, 1.0)
    D = far(torch.zeros((5, N), dtype=TORCH[dtype]), 0)
    lib.gemm_grouped(far(A, 0), B.cuda(), at, out=D)
    done()
    assert_close(D, ref, tol, dtype)
    index = torch.tensor([4, 0, 3, 4, 1], dtype=torch.int32, device="cuda")
    ref, tol, _ = grouped_ref(A, B, off, index, None, 0, 1.0)
    got = lib.gemm_grouped(far(A, 0), far(B, 0), at, row_index=index, out_dtype=torch.float32)
    done()
    assert_close(got, ref, tol, "f32")
    # the other storage order, columns far apart
    Bt = far(B[:1].transpose(1, 2)[:, :5].contiguous(), 1).transpose(1, 2)
    one = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    ref, tol, _ = grouped_ref(A, B[:1, :, :5], np.array([0, 5]), None, None, 0, 1.0)
    got = lib.gemm_grouped(A.cuda(), Bt, one, out_dtype=torch.float32)
    done()
    assert_close(got, ref, tol, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [80, 77])
def test_weight_gradient(dtype, N):
    rng = np.random.default_rng(2)
    sizes, M = [2, 0, 1, 2], 72
    off = offsets_of(sizes)
    at = torch.from_numpy(off).cuda()
    A, B = draw(rng, (5, M), dtype), draw(rng, (5, N), dtype)
    C = torch.from_numpy(rng.standard_normal((4, M, N)).astype(np.float32))
    ref, tol = wgrad_ref(A, B, off, None, C, 1.0, 0.5)
    D = far(torch.zeros((4, M, N)), 0)
    lib.gemm_grouped_wgrad(far(A, 0), far(B, 0), at, C=far(C, 0), beta=0.5, out=D)
    done()
    assert_close(D, ref, tol, "f32")
    ref, tol = wgrad_ref(A[:, :5], B, off, None, None, 1.0, 0.0)
    D = far(torch.zeros((4, 5, N), dtype=TORCH[dtype]), 1)  # rows of D far apart, matrices packed
    lib.gemm_grouped_wgrad(A[:, :5].cuda() if dtype == "f32" else far(A, 0)[:, :5], B.cuda(), at, out=D)
    done()
    assert_close(D, ref, tol, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", [16, 300])
def test_lora(dtype, rank):
    rng = np.random.default_rng(3)
    M, K, N, n = 5, 72, 80, 4
    X, W = draw(rng, (M, K), dtype), draw(rng, (K, N), dtype, sigma=0.1)
    LA, LB = draw(rng, (n, K, rank), dtype, sigma=0.1), draw(rng, (n, rank, N), dtype, sigma=0.1)
    ids = torch.tensor([3, 1, -1, 2, 3], dtype=torch.int32, device="cuda")
    ref, tol = lora_ref(X, W, LA, LB, ids, None, None, 0, dtype, "f32")
    D = far(torch.zeros((M, N)), 0)
    lib.gemm_lora(far(X, 0), W.cuda(), far(LA, 0), far(LB, 0), ids, out=D)
    done()
    assert_close(D, ref, tol, "f32")


CAPTURE = """
import torch
import dense_gemm_08_gb300 as lib
g = torch.Generator(device="cuda").manual_seed(1)
t = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
A, B, G, W, LA, LB = t(96, 64), t(3, 64, 128), t(96, 128), t(64, 128), t(3, 64, 8), t(3, 8, 128)
ids = (torch.arange(96, device="cuda") % 3).to(torch.int32)
off = torch.tensor([0, 30, 31, 96], dtype=torch.int32, device="cuda")
call = lambda: (lib.gemm_grouped(A, B, off), lib.gemm_grouped_wgrad(A, G, off),
                lib.gemm_lora(A, W, LA, LB, ids), lib.gemm_grouped(A.float(), B.float(), off),
                *lib.group_rows(ids, 400))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = call()
graph.replay()
torch.cuda.synchronize()
for a, b in zip(out, call()):
    assert torch.equal(a, b)
assert lib.gemm_last_device_status() == lib.GEMM_OK
"""


def test_first_calls_of_a_process_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([root, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", CAPTURE], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
