"""The adapters' own gradients of gemm_lora, from the grouped operators: with rows
grouped by adapter, U = X LA_a and T = dD LB_a^T are grouped products, and

    dLB_a = s_a U_a^T dD_a,   dLA_a = s_a X_a^T T_a

their weight gradients.  Against the formulas in 64 bits and against central
differences of the library's own forward pass."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import done, draw, padded, rel_sum
from test_gpu_lora import operands

pytestmark = pytest.mark.gpu

UNIT = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def gradients(X, LA, LB, ids, s, G):
    """(dLA, dLB), each a stack like its adapter's matrices."""
    offsets, order, _ = lib.group_rows(ids, LA.shape[0])
    U = lib.gemm_grouped(X, LA, offsets, row_index=order)
    T = lib.gemm_grouped(G, LB.transpose(1, 2), offsets, row_index=order)
    dLB = lib.gemm_grouped_wgrad(G, U, offsets, row_index=order).transpose(1, 2)
    dLA = lib.gemm_grouped_wgrad(X, T, offsets, row_index=order)
    return dLA * s[:, None, None], dLB * s[:, None, None]


def make(dtype, M, K, N, r, n, seed, order=(1, 1, 1)):
    rng = np.random.default_rng(seed)
    X, W, LA, LB = operands(rng, M, K, N, r, n, dtype, order)
    ids = torch.from_numpy(rng.integers(-1, n, M).astype(np.int32)).cuda()
    ids[ids == n - 1] = 0  # an adapter without rows
    s = torch.from_numpy((rng.random(n) + 0.5).astype(np.float32)).cuda()
    G = padded(draw(rng, (M, N), dtype), 8)
    return X, W, LA, LB, ids, s, G


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r,n", [(1, 72, 88, 16, 2), (150, 72, 88, 16, 4), (900, 264, 200, 8, 5),
                                       (33, 200, 136, 24, 40)])
@pytest.mark.parametrize("order", [(1, 1, 1), (0, 0, 0)])
def test_formulas(dtype, M, K, N, r, n, order):
    X, W, LA, LB, ids, s, G = make(dtype, M, K, N, r, n, M, order)
    dLA, dLB = gradients(X, LA, LB, ids, s, G)
    done()
    x, la, lb, g = (t.double() for t in (X, LA, LB, G))
    for a in range(n):
        rows = ids == a
        k = int(rows.sum())
        u, t = x[rows] @ la[a], g[rows] @ lb[a].t()
        su, st = x[rows].abs() @ la[a].abs(), g[rows].abs() @ lb[a].abs().t()
        for got, want, big in ((dLB[a], u.t() @ g[rows], (
                (UNIT[dtype] * u.abs() + rel_sum(K) * su + 2.0 ** -25).t() @ g[rows].abs()
                + rel_sum(k) * u.abs().t() @ g[rows].abs())),
                (dLA[a], x[rows].t() @ t, (
                    x[rows].abs().t() @ (UNIT[dtype] * t.abs() + rel_sum(N) * st + 2.0 ** -25)
                    + rel_sum(k) * x[rows].abs().t() @ t.abs()))):
            off = (got.double() - want * s[a].double()).abs()
            bound = big * s[a].double() * 1.01 + 2.0 ** -22 * want.abs() * s[a].double()
            assert bool((off <= bound).all()), (a, float((off - bound).max()))
            if k == 0:
                assert not bool(got.any())


def test_central_differences():
    """L = sum(G D) is linear in LA and in LB: the quotient has no truncation error.  Steps that
    BF16 holds exactly; what is left is the rounding of the first product (2^-15, an FP32 D) and
    of the sums on one side, of U and T (2^-8) on the other."""
    X, W, LA, LB, ids, s, G = make("bf16", 120, 72, 88, 16, 4, 9)
    rng = np.random.default_rng(10)
    LA.copy_(torch.from_numpy(rng.integers(-3, 4, tuple(LA.shape)).astype(np.float32) / 4))
    LB.copy_(torch.from_numpy(rng.integers(-3, 4, tuple(LB.shape)).astype(np.float32) / 4))
    dLA, dLB = gradients(X, LA, LB, ids, s, G)

    def loss(la, lb):
        D = lib.gemm_lora(X, W, la, lb, ids, scale=s, out_dtype=torch.float32)
        return float((D.double() * G.double()).sum())

    for which, d in (("LA", dLA), ("LB", dLB)):
        t = LA if which == "LA" else LB
        E = torch.from_numpy(rng.integers(-1, 2, tuple(t.shape)).astype(np.float32) / 4).cuda()
        up, down = (t.float() + E).to(t.dtype), (t.float() - E).to(t.dtype)
        assert torch.equal(up.float() - down.float(), 2 * E)
        pair = ((up, LB), (down, LB)) if which == "LA" else ((LA, up), (LA, down))
        quotient = (loss(*pair[0]) - loss(*pair[1])) / 2
        want = float((d.double() * E.double()).sum())
        # sums of absolute values, from the definition
        x, g = X.double().abs(), G.double().abs()
        la, lb = LA.double().abs(), LB.double().abs()
        if which == "LA":
            la = la + E.double().abs()
        else:
            lb = lb + E.double().abs()
        size = float((g * (x @ W.double().abs())).sum()) * rel_sum(72)
        slack = 0.0
        for a in range(4):
            rows = ids == a
            part = (x[rows] @ la[a]) @ lb[a]
            both = float((part * g[rows]).sum()) * float(s[a])
            size += both * (2.0 ** -15 + rel_sum(72) + rel_sum(16))
            slack += both * (2.0 ** -8 + rel_sum(88) + rel_sum(120))
        assert abs(quotient - want) <= size + slack
