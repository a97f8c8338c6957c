"""The grouped products and their weight gradients against their definitions
in 64 bits: types, storage orders, odd sizes, empty groups, gathered rows,
unaligned operands, values that must not be read, streams, graphs."""
import itertools

import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import (D_TYPE, SENTINEL, SUFFIX, TORCH, assert_close, done, draw, grouped_ref,
                             offsets_of, padded, wgrad_ref)

pytestmark = pytest.mark.gpu

RAGGED = [
    # (sizes, rows past the last group)
    ([1], 0),
    ([0, 0, 5, 0], 0),
    ([130, 0, 1, 127, 128, 129], 3),
    ([300, 17, 0, 256, 255, 257, 64, 0], 11),
    ([3] * 45, 0),
]


def stack(rng, groups, K, N, dtype, order, pad, dist="normal"):
    sigma = 1.0 / max(K, 1) ** 0.5
    if order == lib.COL_MAJOR:
        return padded(draw(rng, (groups, N, K), dtype, dist, sigma), pad).transpose(1, 2)
    return padded(draw(rng, (groups, K, N), dtype, dist, sigma), pad)


def run_grouped(rng, sizes, tail, K, N, dtype, order, out, gather=False, bias=False, act=0,
                alpha=1.0, dist="normal", pad=None, pad_d=0, first=0):
    vec = 4 if dtype == "f32" else 8
    pad = vec if pad is None else pad
    rows = first + sum(sizes) + tail
    offsets = offsets_of(sizes, first)
    stored = rows if not gather else max(rows // 2, 1) + 5
    A = padded(draw(rng, (stored, K), dtype, dist), pad)
    B = stack(rng, len(sizes), K, N, dtype, order, pad, dist)
    index = None
    if gather:
        index = torch.from_numpy(rng.integers(0, stored, rows).astype(np.int32)).cuda()
    bias_t = torch.from_numpy(rng.standard_normal((len(sizes), N)).astype(np.float32)).cuda() if bias else None
    buf = torch.full((rows + 2, N + pad_d), SENTINEL, dtype=TORCH[out], device="cuda")
    D = buf[:rows, :N]
    got = lib.gemm_grouped(A, B, torch.from_numpy(offsets).cuda(), row_index=index, bias=bias_t,
                           activation=act, out=D, alpha=alpha)
    name = lib.gemm_last_kernel()
    done()
    ref, tol, inside = grouped_ref(A, B, offsets, index, bias_t, act, alpha)
    what = f"{name} {dtype} sizes {sizes[:8]} K {K} N {N}"
    if dist == "int" and act == 0 and not bias:
        assert np.array_equal(got[torch.from_numpy(inside).cuda()].double().cpu().numpy(), ref[inside]), what
    else:
        assert_close(got[torch.from_numpy(inside).cuda()], ref[inside], tol[inside], out, what)
    left = buf.clone()
    left[:rows, :N][torch.from_numpy(inside).cuda()] = SENTINEL
    assert bool((left == SENTINEL).all()), what + ": a store outside the groups' rows"
    return name


@pytest.mark.parametrize("dtype,order", list(itertools.product(["f32", "bf16", "f16"], [0, 1])))
@pytest.mark.parametrize("ragged", range(len(RAGGED)))
@pytest.mark.parametrize("K,N", [(64, 256), (200, 72), (1, 1), (72, 33), (136, 300)])
def test_grouped_shapes(dtype, order, ragged, K, N):
    sizes, tail = RAGGED[ragged]
    rng = np.random.default_rng(ragged * 100 + K + N + order)
    run_grouped(rng, sizes, tail, K, N, dtype, order, dtype, pad_d=3)


@pytest.mark.parametrize("dtype,order", list(itertools.product(["f32", "bf16", "f16"], [0, 1])))
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_integers_are_exact(dtype, order, gather):
    # partial sums stay below 9 * 136 < 2048: exact in FP32 (and in the FP32 D)
    rng = np.random.default_rng(5 + order)
    run_grouped(rng, [140, 0, 260, 7, 513], 2, 136, 264, dtype, order, "f32", gather=gather,
                dist="int")


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                       ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("act,bias,alpha", [(0, True, 1.0), (1, True, -0.5), (2, True, 1.5),
                                            (2, False, 1.0)])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_epilogue_and_gather(dtype, out, act, bias, alpha, gather):
    rng = np.random.default_rng(act * 10 + gather)
    run_grouped(rng, [200, 3, 0, 129, 310], 5, 264, 392, dtype, act & 1, out, gather=gather,
                bias=bias, act=act, alpha=alpha, pad_d=8)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", [0, 1])
def test_grouped_large_groups(dtype, order):
    # several row tiles per group and column tiles, enough of them for the largest tiles
    rng = np.random.default_rng(77)
    sizes = [1500, 0, 700, 1025] if dtype != "f32" else [700, 0, 300]
    run_grouped(rng, sizes, 0, 512, 4096 if dtype != "f32" else 520, dtype, order,
                "bf16" if dtype == "bf16" else "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", [0, 1])
def test_grouped_unaligned_operands(dtype, order):
    # leading dimensions that TMA cannot describe
    rng = np.random.default_rng(8)
    run_grouped(rng, [70, 0, 130], 1, 77, 51, dtype, order, "f32", pad=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 2, 8, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("order", [0, 1])
def test_grouped_few_rows(dtype, rows, order):
    # a decode step: few rows over more groups than rows
    rng = np.random.default_rng(rows)
    groups = 40
    ids = np.sort(rng.integers(0, groups, rows))
    sizes = np.bincount(ids, minlength=groups).tolist()
    run_grouped(rng, sizes, 0, 520, 264, dtype, order, dtype, gather=rows % 2 == 0)


def test_grouped_first_offset_above_zero_and_many_groups():
    rng = np.random.default_rng(9)
    run_grouped(rng, [4, 0, 150], 9, 64, 64, "bf16", 1, "bf16", first=37)
    sizes = rng.integers(0, 4, 1500).tolist()
    run_grouped(rng, sizes, 0, 40, 48, "bf16", 0, "f32")
    run_grouped(rng, sizes, 0, 40, 48, "f32", 1, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_bad_offsets_and_indexes_stay_in_bounds(dtype):
    # offsets outside [0, rows] are clamped, falling pairs are empty groups,
    # indexes outside A read zeros
    rng = np.random.default_rng(10)
    rows, K, N = 300, 64, 72
    A = draw(rng, (rows, K), dtype).cuda()
    B = stack(rng, 5, K, N, dtype, 1, 8)
    offsets = np.array([-7, 100, 60, 61, 250, 4000], np.int32)
    index = rng.integers(0, rows, rows).astype(np.int32)
    index[[0, 5, 120, 299]] = [-1, rows, 2 ** 31 - 1, -2 ** 31]
    D = torch.full((rows, N), SENTINEL, dtype=torch.float32, device="cuda")
    idx = torch.from_numpy(index).cuda()
    lib.gemm_grouped(A, B, torch.from_numpy(offsets).cuda(), row_index=idx, out=D)
    done()
    # rows 60..100 belong to two groups here: either group's product may be there
    ref, tol, inside = grouped_ref(A, B, offsets, idx, None, 0, 1.0)
    sure = inside.copy()
    sure[60:100] = False
    keep = torch.from_numpy(sure).cuda()
    assert_close(D[keep], ref[sure], tol[sure], "f32")
    assert not bool(torch.isnan(D).any())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_grouped_special_values_stay_in_their_row(dtype):
    rng = np.random.default_rng(11)
    sizes, K, N = [100, 60, 140], 128, 136
    rows = 300
    A = draw(rng, (rows + 40, K), dtype)
    A[rows:] = float("nan")  # rows of no group
    A[99] = float("inf")
    A[130] = float("nan")
    B = draw(rng, (4, N, K), dtype, sigma=0.1)
    B[3] = float("nan")  # a matrix past the last group
    A, B = A.cuda(), B.cuda().transpose(1, 2)[:3]
    offsets = offsets_of(sizes)
    D = torch.zeros((rows + 40, N), dtype=torch.float32, device="cuda")
    lib.gemm_grouped(A, B, torch.from_numpy(offsets).cuda(), out=D)
    done()
    ref, tol, _ = grouped_ref(A, B, offsets, None, None, 0, 1.0)
    ok = np.ones(rows + 40, bool)
    ok[rows:] = ok[99] = ok[130] = False
    assert_close(D[torch.from_numpy(ok).cuda()], ref[ok], tol[ok], "f32")
    assert not bool(torch.isfinite(D[99]).any()) and bool(torch.isnan(D[130]).all())
    assert bool((D[rows:] == 0).all())


def test_grouped_k_zero_and_alpha_zero():
    offsets = torch.tensor([0, 3, 3, 5], dtype=torch.int32, device="cuda")
    bias = torch.arange(3 * 8, dtype=torch.float32, device="cuda").reshape(3, 8) - 10
    for dtype in (torch.float32, torch.bfloat16):
        nan = torch.full((5, 16), float("nan"), dtype=dtype, device="cuda")
        B = torch.full((3, 16, 8), float("nan"), dtype=dtype, device="cuda")
        want = bias[[0, 0, 0, 2, 2]].clamp(min=0)
        got = lib.gemm_grouped(nan, B, offsets, bias=bias, activation=lib.GEMM_ACT_RELU, alpha=0.0)
        assert torch.equal(got.float(), want)
        got = lib.gemm_grouped(nan[:, :0], B[:, :0], offsets, bias=bias,
                               activation=lib.GEMM_ACT_RELU)
        assert torch.equal(got.float(), want)


def run_wgrad(rng, sizes, tail, M, N, dtype, out, gather=False, alpha=1.0, beta=0.0,
              dist="normal", pad=None, pad_d=0, in_place=False, first=0):
    vec = 4 if dtype == "f32" else 8
    pad = vec if pad is None else pad
    rows, groups = first + sum(sizes) + tail, len(sizes)
    offsets = offsets_of(sizes, first)
    stored = rows if not gather else max(rows // 2, 1) + 3
    A = padded(draw(rng, (stored, M), dtype, dist), pad)
    b = draw(rng, (rows, N), dtype, dist)
    # rows of no group must not be read into any result
    b[first + sum(sizes):] = float("nan")
    b[:first] = float("nan")
    B = padded(b, pad)
    index = None
    if gather:
        index = torch.from_numpy(rng.integers(0, stored, rows).astype(np.int32)).cuda()
    buf = torch.full((groups, M + 1, N + pad_d), SENTINEL, dtype=TORCH[out], device="cuda")
    D = buf[:, :M, :N]
    C = None
    if beta:
        C = torch.from_numpy(rng.standard_normal((groups, M, N)).astype(np.float32)).cuda()
        if in_place:
            D.copy_(C)
            C0, C = C, D
    got = lib.gemm_grouped_wgrad(A, B, torch.from_numpy(offsets).cuda(), row_index=index, C=C,
                                 alpha=alpha, beta=beta, out=D)
    name = lib.gemm_last_kernel()
    done()
    ref, tol = wgrad_ref(A, B, offsets, index, C0 if in_place else C, alpha, beta)
    what = f"{name} {dtype} sizes {sizes[:8]} M {M} N {N}"
    if dist == "int" and not beta:
        assert np.array_equal(got.double().cpu().numpy(), ref), what
    else:
        assert_close(got, ref, tol, out, what)
    left = buf.clone()
    left[:, :M, :N] = SENTINEL
    assert bool((left == SENTINEL).all()), what + ": a store outside D"
    return name


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ragged", range(len(RAGGED)))
@pytest.mark.parametrize("M,N", [(128, 256), (72, 200), (1, 1), (33, 72), (300, 136)])
def test_wgrad_shapes(dtype, ragged, M, N):
    sizes, tail = RAGGED[ragged]
    run_wgrad(np.random.default_rng(ragged * 100 + M + N), sizes, tail, M, N, dtype, dtype,
              pad_d=3)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gather", [False, True])
def test_wgrad_integers_are_exact(dtype, gather):
    # |sum| <= 9 * 513 < 2^24; every row-count remainder modulo the block of 64 and the slice of 16
    rng = np.random.default_rng(15)
    run_wgrad(rng, [513, 0, 1, 15, 16, 17, 63, 64, 65, 80, 81, 127, 128], 2, 264, 136, dtype,
              "f32", gather=gather, dist="int")


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"),
                                       ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("alpha,beta,in_place", [(1.0, 0.0, False), (0.5, 1.0, False),
                                                 (-1.0, -0.25, True)])
def test_wgrad_accumulates(dtype, out, gather, alpha, beta, in_place):
    if in_place and out != "f32":
        in_place = False
    run_wgrad(np.random.default_rng(16), [200, 0, 70, 333], 4, 200, 328, dtype, out,
              gather=gather, alpha=alpha, beta=beta, pad_d=8, in_place=in_place)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wgrad_unaligned_operands(dtype):
    run_wgrad(np.random.default_rng(17), [70, 0, 130], 1, 77, 51, dtype, "f32", pad=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_wgrad_large(dtype):
    sizes = [900, 0, 1300, 65] if dtype != "f32" else [300, 0, 200]
    M, N = (1024, 4096) if dtype != "f32" else (264, 520)
    run_wgrad(np.random.default_rng(18), sizes, 0, M, N, dtype, "f32", first=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_wgrad_special_values_stay_in_their_group(dtype):
    rng = np.random.default_rng(19)
    sizes, M, N = [67, 30, 100], 72, 80
    a, b = draw(rng, (197, M), dtype), draw(rng, (197, N), dtype)
    a[70], b[75] = float("nan"), float("inf")  # group 1
    A, B = a.cuda(), b.cuda()
    offsets = offsets_of(sizes)
    got = lib.gemm_grouped_wgrad(A, B, torch.from_numpy(offsets).cuda())
    done()
    ref, tol = wgrad_ref(A, B, offsets, None, None, 1.0, 0.0)
    for g in (0, 2):
        assert_close(got[g], ref[g], tol[g], "f32")
    assert bool(torch.isnan(got[1]).all())


def test_wgrad_without_rows_gives_beta_c():
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    C = torch.randn(3, 40, 24, device="cuda")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        A = torch.zeros((0, 40), dtype=dtype, device="cuda")
        B = torch.zeros((0, 24), dtype=dtype, device="cuda")
        assert torch.equal(lib.gemm_grouped_wgrad(A, B, offsets, C=C, beta=0.5), 0.5 * C)
        out = torch.full((3, 40, 24), float("nan"), device="cuda")
        lib.gemm_grouped_wgrad(A, B, offsets, out=out)
        assert bool((out == 0).all())
        # alpha = 0: A and B are not read
        A = torch.full((9, 40), float("nan"), dtype=dtype, device="cuda")
        B = torch.full((9, 24), float("nan"), dtype=dtype, device="cuda")
        some = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")
        assert torch.equal(lib.gemm_grouped_wgrad(A, B, some, C=C, alpha=0.0, beta=1.0), C)


def test_gradients_match_the_formula_and_differences():
    """L = sum(G * D) of the grouped product: its gradients from the library
    against the formulas in 64 bits and against central differences of the
    library's own forward pass (FP32; L is linear in A and in B, so the
    difference quotient has no truncation error, only L's rounding)."""
    rng = np.random.default_rng(20)
    sizes, K, N = [40, 0, 75, 9], 60, 52
    offsets = torch.from_numpy(offsets_of(sizes)).cuda()
    rows = sum(sizes)
    A = draw(rng, (rows, K), "f32").cuda()
    B = draw(rng, (4, K, N), "f32", sigma=0.2).cuda()
    G = draw(rng, (rows, N), "f32").cuda()
    dA = lib.gemm_grouped(G, B.transpose(1, 2), offsets)
    dB = lib.gemm_grouped_wgrad(A, G, offsets)
    done()
    refA, tolA, _ = grouped_ref(G, B.transpose(1, 2), offsets.cpu().numpy(), None, None, 0, 1.0)
    refB, tolB = wgrad_ref(A, G, offsets.cpu().numpy(), None, None, 1.0, 0.0)
    assert_close(dA, refA, tolA, "f32")
    assert_close(dB, refB, tolB, "f32")

    def loss(a, b):
        return float((lib.gemm_grouped(a, b, offsets).double() * G.double()).sum())

    h = 0.5
    for x, dx, f in ((A, dA, lambda e: loss(A + e, B)), (B, dB, lambda e: loss(A, B + e))):
        E = torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)).cuda()
        quotient = (f(h * E) - f(-h * E)) / (2 * h)
        # rounding: both losses are sums of rows * N terms |G D| off by at most K 2^-24 of
        # their absolute sums; x + h E adds 2^-24 relative
        size = float((G.double().abs() * lib.gemm_grouped(
            (A.abs() + E.abs() if x is A else A.abs()),
            (B.abs() + E.abs() if x is B else B.abs()), offsets).double()).sum())
        assert abs(quotient - float((dx.double() * E.double()).sum())) <= 2 * (K + 4) * 2.0 ** -24 * size / h


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_grouped_streams_graphs_and_repeats(dtype):
    rng = np.random.default_rng(21)
    sizes, K, N = [300, 40, 0, 260], 200, 264
    offsets = torch.from_numpy(offsets_of(sizes)).cuda()
    A = padded(draw(rng, (600, K), dtype), 8)
    B = stack(rng, 4, K, N, dtype, 1, 8)
    G = padded(draw(rng, (600, N), dtype), 8)
    first = (lib.gemm_grouped(A, B, offsets), lib.gemm_grouped_wgrad(A, G, offsets))
    done()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = (lib.gemm_grouped(A, B, offsets), lib.gemm_grouped_wgrad(A, G, offsets))
    side.synchronize()
    for x, y in zip(first, again):
        assert torch.equal(x, y)  # the same bits on every run
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = (lib.gemm_grouped(A, B, offsets), lib.gemm_grouped_wgrad(A, G, offsets))
    # other sizes, found by the replayed kernels on the device
    new = offsets_of([10, 290, 299, 1])
    offsets.copy_(torch.from_numpy(new))
    graph.replay()
    done()
    ref, tol, _ = grouped_ref(A, B, new, None, None, 0, 1.0)
    assert_close(out[0], ref, tol, dtype)
    ref, tol = wgrad_ref(A, G, new, None, None, 1.0, 0.0)
    assert_close(out[1], ref, tol, "f32")


def test_grouped_one_matrix_for_all_groups():
    # stride_b = 0, through the C entry points' arguments
    rng = np.random.default_rng(22)
    for dtype in ("f32", "bf16", "f16"):
        A = draw(rng, (90, 64), dtype).cuda()
        B = draw(rng, (1, 64, 72), dtype).cuda()
        offsets = torch.from_numpy(offsets_of([20, 0, 70])).cuda()
        D = torch.zeros((90, 72), dtype=torch.float32, device="cuda")
        getattr(lib, "gemm_grouped_" + SUFFIX[dtype])(
            3, 90, 72, 64, 1.0, A, 64, 90, None, offsets, B, 72, 0, lib.ROW_MAJOR, D, 72,
            d_type=D_TYPE["f32"])
        done()
        ref, tol, _ = grouped_ref(A, B.expand(3, 64, 72), offsets.cpu().numpy(), None, None, 0, 1.0)
        assert_close(D, ref, tol, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_grouped_stacks_interleaved_and_broadcast(dtype):
    # matrices of a stack that share rows of one buffer (pitch groups * N, matrix pitch N),
    # and a C that is the same for all groups
    rng = np.random.default_rng(23)
    sizes, K, N = [70, 0, 33], 64, 72
    offsets = offsets_of(sizes)
    at = torch.from_numpy(offsets).cuda()
    A = draw(rng, (103, K), dtype).cuda()
    B = draw(rng, (K, 3, N), dtype, sigma=0.1).cuda().permute(1, 0, 2)
    got = lib.gemm_grouped(A, B, at, out_dtype=torch.float32)
    done()
    ref, tol, _ = grouped_ref(A, B, offsets, None, None, 0, 1.0)
    assert_close(got, ref, tol, "f32")
    G = draw(rng, (103, N), dtype).cuda()
    C = torch.from_numpy(rng.standard_normal((1, K, N)).astype(np.float32)).cuda().expand(3, K, N)
    buf = torch.full((K + 1, 3, N), SENTINEL, dtype=torch.float32, device="cuda")
    lib.gemm_grouped_wgrad(A, G, at, C=C, beta=2.0, out=buf[:K].permute(1, 0, 2))
    done()
    ref, tol = wgrad_ref(A, G, offsets, None, C, 1.0, 2.0)
    assert_close(buf[:K].permute(1, 0, 2), ref, tol, "f32")
    assert bool((buf[K] == SENTINEL).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N", [248, 250, 251])
@pytest.mark.parametrize("M", [200, 256])
def test_wgrad_rows_of_any_alignment(dtype, N, M):
    # rows of D and C on 16, 8 and 2 bytes; few and many rows per group (boxes, registers)
    for sizes in ([40, 0, 90], [1500, 700]):
        rng = np.random.default_rng(24 + N)
        run_wgrad(rng, sizes, 3, M, N, dtype, dtype, beta=1.0)
        run_wgrad(rng, sizes, 3, M, N, dtype, "f32")
