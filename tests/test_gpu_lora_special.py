"""gemm_lora with infinities and NaNs: a row's result is what the definition
makes of its own row of X, of W and of its own adapter, whatever the adapters of
the rows beside it hold, and one such row does not hold up the others."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH, done, f64, lora_ref
from test_gpu_lora import operands

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
OUT = [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]


def definition(X, W, LA, LB, ids):
    """act = none, scale = 1; the value itself in 64 bits, infinities and NaNs included."""
    x, w, la, lb = f64(X), f64(W), f64(LA), f64(LB)
    with np.errstate(invalid="ignore"):
        z = x @ w
        # (a library product may skip zeros: the rows and columns that matter are summed plainly)
        for i in np.flatnonzero(~np.isfinite(x).all(1)):
            z[i] = (x[i][:, None] * w).sum(0)
        for j in np.flatnonzero(~np.isfinite(w).all(0)):
            z[:, j] = (x * w[:, j]).sum(1)
        for i, a in enumerate(ids.cpu().numpy()):
            if 0 <= a < la.shape[0]:
                u = (x[i][:, None] * la[a]).sum(0)
                z[i] += (u[:, None] * lb[a]).sum(0)
    return z


def check(X, W, LA, LB, ids, dtype, out):
    D = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=TORCH[out])
    done()
    got, want = f64(D), definition(X, W, LA, LB, ids)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    finite = np.isfinite(want)
    clean = [torch.nan_to_num(t, nan=0.0, posinf=0.0, neginf=0.0) for t in (X, W, LA, LB)]
    _, tol = lora_ref(*clean, ids, None, None, 0, dtype, out)
    unit = {"f32": 2.0 ** -22, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out]
    off = np.abs(got[finite] - want[finite])
    assert bool((off <= tol[finite] * (1 + 2.0 ** -8) + unit * np.abs(want[finite]) + 2.0 ** -24).all())


def case(seed, M, dtype, order, K=200, N=300, rank=16):
    rng = np.random.default_rng(seed)
    n = 6
    X, W, LA, LB = operands(rng, M, K, N, rank, n, dtype, order)
    ids = torch.from_numpy((np.arange(M) % (n + 1) - 1).astype(np.int32)).cuda()
    return X, W, LA, LB, ids


@pytest.mark.parametrize("dtype,out", OUT)
@pytest.mark.parametrize("M", [1, 20, 70, 300])
@pytest.mark.parametrize("order", [(1, 1, 1), (0, 0, 0)])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
def test_in_a_row_and_a_column(dtype, out, M, order, value):
    X, W, LA, LB, ids = case(M, M, dtype, order)
    X[0, 3] = value                # a row without an adapter
    X[M // 2, 199] = value
    W[77, 5], W[1, 299] = value, value
    check(X, W, LA, LB, ids, dtype, out)


@pytest.mark.parametrize("dtype,out", OUT)
@pytest.mark.parametrize("M", [20, 70, 300])
@pytest.mark.parametrize("order", [(1, 1, 1), (0, 0, 0), (1, 1, 0)])
def test_in_one_and_in_several_adapters(dtype, out, M, order):
    X, W, LA, LB, ids = case(M + 1, M, dtype, order)
    LB[2, 3, 5], LB[2, 4, 299], LB[2, 0, 40] = INF, NAN, -INF
    check(X, W, LA, LB, ids, dtype, out)
    LB[4, :, 260:] = NAN
    LB[1, 15, 299] = INF
    check(X, W, LA, LB, ids, dtype, out)
    LA[3, 100, 7] = NAN
    X[5, 8], X[6, 9] = NAN, INF
    W[0, 5], W[0, 6] = INF, NAN
    check(X, W, LA, LB, ids, dtype, out)


@pytest.mark.parametrize("dtype,out", OUT)
@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("rank", [1, 4, 24, 40])
@pytest.mark.parametrize("order", [(1, 1, 1), (0, 0, 0)])
def test_ranks_between_powers_of_two(dtype, out, M, rank, order):
    # (the kernels pad them with zeros, which infinities must not meet)
    X, W, LA, LB, ids = case(M + rank, M, dtype, order, rank=rank)
    X[5, 8], X[6, 9], X[7, 10], X[13, 199] = INF, -INF, INF, NAN
    check(X, W, LA, LB, ids, dtype, out)
    LB[2, 0, 5] = INF
    check(X, W, LA, LB, ids, dtype, out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sums_in_parts(dtype):
    for M in (9, 200):
        X, W, LA, LB, ids = case(M, M, dtype, (1, 1, 1), K=1600, N=520)
        LB[2, 3, 5], LB[0, 4, 519], LB[5, 0] = INF, NAN, -INF
        X[4, 1000] = NAN
        X[8, 1500] = INF
        W[700, 100] = NAN
        check(X, W, LA, LB, ids, dtype, "f32")


def test_with_bias_and_activation():
    X, W, LA, LB, ids = case(7, 70, "bf16", (1, 1, 1))
    LB[2, 3], LB[3, 4, 17] = INF, NAN
    bias = torch.linspace(-2, 2, 300, device="cuda")
    for act in (lib.GEMM_ACT_RELU, lib.GEMM_ACT_GELU):
        for out in ("bf16", "f32"):
            D = lib.gemm_lora(X, W, LA, LB, ids, bias=bias, activation=act, out_dtype=TORCH[out])
            done()
            keep = ((ids != 2) & (ids != 3)).cpu().numpy()
            clean = LB.clone()
            clean[2:4] = 0
            ref, tol = lora_ref(X, W, LA, clean, ids, None, bias, act, "bf16", out)
            got = f64(D)[keep]
            unit = 2.0 ** -8 if out == "bf16" else 2.0 ** -22
            assert bool((np.abs(got - ref[keep]) <= tol[keep] * 1.01 + unit * np.abs(ref[keep])).all())


def median_us(call, n=9):
    times = []
    for _ in range(n + 2):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times[2:])[n // 2]


@pytest.mark.parametrize("where", ["X", "X without adapter", "W"])
def test_bad_requests_do_not_hold_up_their_batch(where):
    # half the rows hold a NaN, or a column of W does: nothing is there to compute again
    M, K, N, n = 64, 8192, 2048, 8
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, 0.1, generator=g)

    X, W = normal(M, K), normal(N, K).t()
    LA, LB = normal(n, 16, K).transpose(1, 2), normal(n, N, 16).transpose(1, 2)
    ids = (torch.arange(M, device="cuda") % (n + 1) - 1).to(torch.int32)
    call = lambda: lib.gemm_lora(X, W, LA, LB, ids)  # noqa: E731
    clean = median_us(call)
    if where == "X":
        X[ids.cpu() % 2 == 1, 17] = NAN
    elif where == "W":
        W[9, 77] = NAN
    else:
        X[ids.cpu() < 0, 17] = NAN
    bad = median_us(call)
    done()
    assert bad <= 8 * clean + 50, (bad, clean)


def test_a_tile_of_sums_computed_again_within_the_waits():
    # every sum of the tile's other rows depends on another adapter's infinities
    M, K, N = 128, 49152, 256
    X = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((K, N), dtype=torch.bfloat16, device="cuda")
    LA = torch.ones((2, K, 8), dtype=torch.bfloat16, device="cuda")
    LB = torch.ones((2, 8, N), dtype=torch.bfloat16, device="cuda")
    LB[1] = INF
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    ids[5] = 1
    D = lib.gemm_lora(X, W, LA, LB, ids, out_dtype=torch.float32)
    done()
    assert bool(torch.isinf(D[5]).all())
    D[5] = K + 8.0 * K
    assert bool((D == K + 8.0 * K).all())


@pytest.mark.parametrize("dtype,out", OUT)
def test_tiles_of_two_ctas(dtype, out):
    X, W, LA, LB, ids = case(3, 2600, dtype, (1, 1, 1), K=136, N=2600, rank=20)
    X[5, 8], X[1300, 9], X[2599, 135] = INF, NAN, -INF
    W[7, 2000] = INF
    LB[2, 3, 5], LB[4, 0, 1000], LB[1, 19, 2599] = INF, NAN, -INF
    check(X, W, LA, LB, ids, dtype, out)
    assert lib.gemm_last_kernel().endswith("pair>")
