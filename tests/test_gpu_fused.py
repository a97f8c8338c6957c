"""The fused products and their gradients against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH, f64
from mixture_harness import check, fused_grad_ref, fused_ref, stored

pytestmark = pytest.mark.gpu
NONE, RELU, GELU, SILU = (lib.GEMM_ACT_NONE, lib.GEMM_ACT_RELU, lib.GEMM_ACT_GELU, lib.GEMM_ACT_SILU)


def operand(rng, r, c, dtype, order, extra, sigma=1.0):
    """r x c, row- or column-major, its stored rows padded."""
    x = rng.standard_normal((r, c)) * sigma
    return stored(x, dtype, extra) if order == 0 else stored(x.T, dtype, extra).t()


def pad_for(c, dtype, aligned):
    """Padding that starts rows on 16 bytes, or does not."""
    vec = 4 if dtype == "f32" else 8
    return (-c) % vec if aligned else (-c) % vec + 1


SIZES = [(1, 1, 1), (1, 64, 64), (1, 300, 515), (2, 130, 1000), (3, 17, 4096), (4, 257, 96), (5, 64, 128),
         (17, 40, 33), (64, 256, 192), (100, 300, 71), (129, 257, 130), (200, 520, 640), (300, 1030, 65)]


def run_fused(M, N, K, dtype, oa, ob, act, bias, residual, pre, aligned=True, alpha=1.0, seed=0):
    rng = np.random.default_rng([M, N, K, seed])
    A = operand(rng, M, K, dtype, oa, pad_for(M if oa else K, dtype, aligned))
    B = operand(rng, K, N, dtype, ob, pad_for(K if ob else N, dtype, aligned), max(K, 1) ** -0.5)
    extra = pad_for(N, dtype, aligned)
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).cuda() if bias else None
    R = stored(rng.standard_normal((M, N)), dtype, extra) if residual else None
    out = stored(np.full((M, N), 3.0), dtype, extra + 8, fill=5.0)
    got = lib.gemm_fused(A, B, bias=b, activation=act, residual=R, keep_pre=pre, alpha=alpha, out=out)
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    z = None
    if pre:
        got, z = got
    d, dtol, zr, ztol = fused_ref(A, B, b, act, R, alpha, dtype)
    check(got, d, dtol, "D")
    if pre:
        check(z, zr, ztol, "Z")
    whole = out.as_strided((M, N + extra + 8), out.stride(), out.storage_offset())
    assert (whole[:, N:] == 5.0).all()
    return A, B, b, R, got


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sizes(dtype, aligned, M, N, K):
    for oa, ob in ((0, 1), (0, 0), (1, 0), (1, 1)):
        run_fused(M, N, K, dtype, oa, ob, GELU, True, True, False, aligned)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 4, 50, 300])
@pytest.mark.parametrize("act", [NONE, RELU, GELU, SILU])
@pytest.mark.parametrize("bias,residual,pre", [(False, False, False), (True, False, True),
                                               (False, True, True), (True, True, False),
                                               (True, True, True)])
def test_what_follows_the_product(dtype, M, act, bias, residual, pre):
    run_fused(M, 200, 136, dtype, 0, 1, act, bias, residual, pre, alpha=1.5)


def run_grad(M, N, K, dtype, oa, ob, act, dbias, aligned=True, alpha=1.0, seed=0):
    rng = np.random.default_rng([M, N, K, seed, 9])
    A = operand(rng, M, K, dtype, oa, pad_for(M if oa else K, dtype, aligned))
    B = operand(rng, K, N, dtype, ob, pad_for(K if ob else N, dtype, aligned), max(K, 1) ** -0.5)
    extra = pad_for(N, dtype, aligned)
    Z = stored(rng.standard_normal((M, N)) * 1.5, dtype, extra)
    out = stored(np.full((M, N), 3.0), dtype, extra + 8, fill=5.0)
    got = lib.gemm_fused_grad(A, B, Z, activation=act, bias_grad=dbias, alpha=alpha, out=out)
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    d, dtol, s, stol = fused_grad_ref(A, B, Z, act, alpha, dtype)
    if dbias:
        got, sums = got
        check(sums, s, stol, "dbias")
    check(got, d, dtol, "D")
    whole = out.as_strided((M, N + extra + 8), out.stride(), out.storage_offset())
    assert (whole[:, N:] == 5.0).all()
    over = Z.clone()
    again = lib.gemm_fused_grad(A, B, over, activation=act, alpha=alpha, bias_grad=dbias, out=over)
    assert torch.equal(again[0] if dbias else again, got)
    # (without the column sums a long K is summed another way)
    check(lib.gemm_fused_grad(A, B, Z, activation=act, alpha=alpha), d, dtol, "D alone")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gradient_sizes(dtype, aligned, M, N, K):
    for oa, ob in ((0, 0), (0, 1), (1, 0)):
        run_grad(M, N, K, dtype, oa, ob, GELU, True, aligned)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 4, 50, 300])
@pytest.mark.parametrize("act", [NONE, RELU, GELU, SILU])
@pytest.mark.parametrize("dbias", [False, True])
def test_gradient_activations(dtype, M, act, dbias):
    run_grad(M, 200, 136, dtype, 0, 0, act, dbias, alpha=0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_no_steps_of_k_and_alpha_zero(dtype):
    t = TORCH[dtype]
    A, B = torch.zeros(5, 0, dtype=t, device="cuda"), torch.zeros(0, 24, dtype=t, device="cuda")
    b = torch.randn(24, device="cuda")
    R = torch.randn(5, 24, device="cuda").to(t)
    want, tol, z, ztol = fused_ref(A, B, b, SILU, R, 1.0, dtype)
    check(lib.gemm_fused(A, B, bias=b, activation=SILU, residual=R), want, tol)
    nan = torch.full((5, 16), float("nan"), dtype=t, device="cuda")
    got = lib.gemm_fused(nan, nan[:, :1].expand(5, 24).contiguous()[:1].expand(16, 24).contiguous(),
                         bias=b, activation=SILU, residual=R, alpha=0.0)  # A and B are not read
    check(got, want, tol)
    d, s = lib.gemm_fused_grad(A, B, R, activation=SILU, bias_grad=True)
    assert (d == 0).all() and (s == 0).all()
    d, s = lib.gemm_fused_grad(torch.zeros(0, 16, dtype=t, device="cuda"),
                               torch.zeros(16, 24, dtype=t, device="cuda"),
                               torch.zeros(0, 24, dtype=t, device="cuda"), activation=GELU,
                               bias_grad=True)
    assert d.shape == (0, 24) and (s == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_special_values(dtype, M):
    """A row's NaNs and infinities stay in it; activations and slopes at the ends of their range."""
    rng = np.random.default_rng(M)
    t = TORCH[dtype]
    A = torch.from_numpy(rng.standard_normal((M, 64))).to(t).cuda()
    B = torch.from_numpy(rng.standard_normal((64, 48))).to(t).cuda()
    clean = lib.gemm_fused(A, B, activation=GELU)
    bad = A.clone()
    bad[M // 2, 3] = float("nan")
    for act in (RELU, GELU, SILU):
        got = lib.gemm_fused(bad, B, activation=act)
        assert torch.isnan(got[M // 2]).all()
        rest = [i for i in range(M) if i != M // 2]
        if act == GELU:
            assert torch.equal(got[rest], clean[rest])
    big = 60000.0 if dtype == "f16" else 1e30
    Z = torch.zeros(M, 48, device="cuda")
    Z[:, 0::6], Z[:, 1::6], Z[:, 2::6] = big, -big, float("inf")
    Z[:, 3::6], Z[:, 4::6], Z[:, 5::6] = float("-inf"), float("nan"), -20.0
    Z = Z.to(t)
    one = lib.gemm_fused_grad(A, B, None, activation=NONE)
    for act in (RELU, GELU, SILU):
        d = lib.gemm_fused_grad(A, B, Z, activation=act)
        assert torch.equal(d[:, 0::6], one[:, 0::6]) and torch.equal(d[:, 2::6], one[:, 2::6])
        assert (d[:, 1::6] == 0).all() and (d[:, 3::6] == 0).all()
        assert torch.isnan(d[:, 4::6]).all()
        assert (d[:, 5::6].float().abs() < 1e-6 * (1 + one[:, 5::6].float().abs()) * 40).all()
    # activations of values past every range: 0 and x
    C = torch.zeros(1, 2, device="cuda")
    for act in (RELU, GELU, SILU):
        y = lib.gemm_fused(torch.zeros(1, 8, dtype=t, device="cuda"),
                           torch.zeros(8, 2, dtype=t, device="cuda"),
                           bias=torch.tensor([-big, big], device="cuda"), activation=act)
        assert y[0, 0] == 0 and y[0, 1] == torch.tensor(big).to(t)
    del C


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slopes_against_differences(dtype):
    """D over a product of ones is act'(Z): central differences of the activation in 64 bits."""
    from mixture_harness import activation
    z = torch.linspace(-13, 13, 400).to(TORCH[dtype])
    h = 1e-5
    for act in (GELU, SILU):
        x = z.double().numpy()
        ref = (activation(x + h, act) - activation(x - h, act)) / (2 * h)
        got = lib.gemm_fused_grad(torch.ones(2, 1, dtype=TORCH[dtype], device="cuda"),
                                  torch.ones(1, 400, dtype=TORCH[dtype], device="cuda"),
                                  z.cuda()[None].expand(2, 400).contiguous(), activation=act)
        tol = np.abs(ref) * (2.0 ** -8 if dtype == "bf16" else 0) + 2.0 ** -18 + 1e-9
        check(got, np.broadcast_to(ref, (2, 400)), np.broadcast_to(tol, (2, 400)))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [2, 200])
def test_streams_graphs_and_in_place(dtype, M):
    t = TORCH[dtype]
    A, B = torch.randn(M, 128, device="cuda").to(t), torch.randn(128, 96, device="cuda").to(t)
    R = torch.randn(M, 96, device="cuda").to(t)
    want = lib.gemm_fused(A, B, residual=R, activation=SILU)
    dw, sw = lib.gemm_fused_grad(A, B, R, activation=GELU, bias_grad=True)
    over = R.clone()
    assert torch.equal(lib.gemm_fused(A, B, residual=over, activation=SILU, out=over), want)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [lib.gemm_fused(A, B, residual=R, activation=SILU, stream=s) for s in sides]
    grads = [lib.gemm_fused_grad(A, B, R, activation=GELU, bias_grad=True, stream=s) for s in sides]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    assert all(torch.equal(d, dw) and torch.equal(s, sw) for d, s in grads)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d = lib.gemm_fused(A, B, residual=R, activation=SILU)
            g, s = lib.gemm_fused_grad(A, B, R, activation=GELU, bias_grad=True)
        graphs.append((graph, d, g, s))
    for (graph, *_), side in zip(graphs, sides):  # side by side
        with torch.cuda.stream(side):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for _, d, g, s in graphs:
        assert torch.equal(d, want) and torch.equal(g, dw) and torch.equal(s, sw)


def test_offsets_past_32_bits():
    """Rows of every matrix more than 2^31 elements apart."""
    pitch = (1 << 30) + 8
    rng = np.random.default_rng(0)

    def far(x):
        t = torch.empty(2 * pitch + x.shape[1], dtype=torch.bfloat16, device="cuda")
        v = t.as_strided((3, x.shape[1]), (pitch, 1))
        v.copy_(x)
        return v

    A = torch.from_numpy(rng.standard_normal((3, 64))).bfloat16().cuda()
    B = torch.from_numpy(rng.standard_normal((64, 40))).bfloat16().cuda()
    R = torch.from_numpy(rng.standard_normal((3, 40))).bfloat16().cuda()
    want = lib.gemm_fused(A, B, residual=R, activation=SILU)
    fa = far(A)
    got = lib.gemm_fused(fa, B, residual=R, activation=SILU, out=far(R))
    assert torch.equal(got.contiguous(), want)
    del fa, got
    wd, ws = lib.gemm_fused_grad(A, B, R, activation=GELU, bias_grad=True)
    fz = far(R)
    gd, gs = lib.gemm_fused_grad(A, B, fz, activation=GELU, bias_grad=True, out=fz)
    assert torch.equal(gd.contiguous(), wd) and torch.equal(gs, ws)
    del fz, gd
    Bt = far(torch.from_numpy(rng.standard_normal((3, 64))).bfloat16().cuda())  # 3 columns, far apart
    assert torch.equal(lib.gemm_fused(A, Bt.t()), lib.gemm_fused(A, Bt.contiguous().t()))


# ------------------------------------------------- larger products, each way they are cut
def big(M, N, K, dtype, oa, ob, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = TORCH[dtype]

    def normal(r, c, order, sigma=1.0):
        if order:
            return normal(c, r, 0, sigma).t()
        ld = -(-c // 8) * 8
        return torch.empty(r, ld, device="cuda", dtype=t).normal_(0, sigma, generator=g)[:, :c]

    return (normal(M, K, oa), normal(K, N, ob, K ** -0.5), normal(M, N, 0), normal(M, N, 0),
            torch.randn(N, device="cuda", generator=g))


def near(got, ref, size, K, dtype, steep=1.0, extra=0.0):
    """Within the sums' bound (rel_sum(K) of `size`), the epilogue's and half a step of the type."""
    from grouped_harness import rel_sum
    from mixture_harness import HALF_STEP, LEAST
    tol = steep * rel_sum(K) * size + 2.0 ** -20 * ref.abs() + 2.0 ** -19 + extra
    tol = tol * (1 + HALF_STEP[dtype]) + ref.abs() * HALF_STEP[dtype] + LEAST[dtype]
    off = (got.double() - ref).abs()
    assert (off <= tol).all(), f"{int((off > tol).sum())} off, worst {float((off / tol).max()):.3g}"


# (None: whichever the library's model of their times picks)
CUTS = [("fused_tc<{},pair>", 2300, 4100, 4096), ("fused_tc<{},pair>", 4097, 8200, 1000), (None, 4097, 2305, 72),
        (None, 600, 9000, 328), (None, 2100, 2500, 200),
        ("fused_tc<{}>", 100, 9001, 264), ("fused_tc<{}>", 40, 20000, 512), ("fused_tc<{}>", 9, 12345, 64),
        ("fused_tc<{}>", 7, 1000, 640), (None, 64, 4096, 4096), (None, 120, 14336, 1024),
        ("fused_tc<{},split>", 64, 1000, 8192), ("fused_tc<{},split>", 16, 200, 8192),
        ("fused_tc<{},split>", 33, 64, 8000), (None, 33, 64, 1000), (None, 256, 515, 2048), (None, 130, 9001, 264),
        (None, 500, 300, 3000), (None, 300, 130, 9000)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("oa,ob", [(0, 1), (0, 0), (1, 0)])
@pytest.mark.parametrize("kernel,M,N,K", CUTS)
def test_cuts(dtype, oa, ob, kernel, M, N, K):
    A, B, R, Z, b = big(M, N, K, dtype, oa, ob)
    z = A.double() @ B.double()
    size = A.double().abs() @ B.double().abs()
    got, pre = lib.gemm_fused(A, B, bias=b, activation=SILU, residual=R, keep_pre=True)
    name = lib.gemm_last_kernel()
    if kernel is not None and not oa:  # (an M-major A has 128 rows per tile)
        assert name == kernel.format(dtype)
    near(pre, z + b.double(), size, K, dtype)
    ref = torch.nn.functional.silu(z + b.double()) + R.double()
    near(got, ref, size, K, dtype, 1.13)
    only = lib.gemm_fused(A, B)
    near(only, z, size, K, dtype)
    d, sums = lib.gemm_fused_grad(A, B, Z, activation=GELU, bias_grad=True)
    x = Z.double().requires_grad_()
    torch.nn.functional.gelu(x, approximate="tanh").sum().backward()
    ref = z * x.grad
    near(d, ref, size, K, dtype, 1.13, 2.0 ** -18 * z.abs())
    from grouped_harness import rel_sum
    tol = ((1.13 * rel_sum(K) * size).sum(0) + (2.0 ** -18 * z.abs()).sum(0) +
           200 * 2.0 ** -24 * ref.abs().sum(0))
    assert ((sums.double() - ref.sum(0)).abs() <= tol).all()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
    # the same bits every time, whatever the matrices' alignment
    again, sums2 = lib.gemm_fused_grad(A, B, Z, activation=GELU, bias_grad=True)
    assert torch.equal(again, d) and torch.equal(sums, sums2)
    odd = torch.empty(M, N + 3, dtype=A.dtype, device="cuda")[:, 1:N + 1]
    zo = torch.empty(M, N + 5, dtype=A.dtype, device="cuda")[:, 2:N + 2]
    zo.copy_(Z)
    again, sums2 = lib.gemm_fused_grad(A, B, zo, activation=GELU, bias_grad=True, out=odd)
    assert torch.equal(again, d) and torch.equal(sums, sums2)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("oa,ob", [(0, 0), (0, 1), (1, 0)])
@pytest.mark.parametrize("kernel,M,N,K", [("fused_tc<{},pair>", 2300, 2600, 6000), ("fused_tc<{}>", 500, 1100, 14336),
                                          ("fused_tc<{}>", 130, 1030, 20001), (None, 64, 300, 4100),
                                          (None, 1, 64, 30000), (None, 2000, 30, 2049),
                                          (None, 700, 1500, 776)])
def test_column_sums_of_a_long_k(dtype, oa, ob, kernel, M, N, K):
    """Sums in parts.  An addition to the accumulator cuts half a unit of its last place on the mean, 0.36 *
    2^-23 of it; sixteen products enter at once, and a random sum's size on the way is 2/3 of its last: 1.8e-9 per
    step of K, that is 1.4e-6 for a part of 768 and 3.7e-6 for a cluster's piece of 2048 (3.6e-5 for the longest
    K here, if it were not cut).  Twice that, and 1e-6 for the rest."""
    A, B, _, Z, _ = big(M, N, K, dtype, oa, ob, seed=3)
    z = A.double() @ B.double()
    size = A.double().abs() @ B.double().abs()
    for act in (NONE, GELU):
        d, sums = lib.gemm_fused_grad(A, B, Z, activation=act, bias_grad=True)
        name = lib.gemm_last_kernel()
        if kernel is not None and not oa and K % 8 == 0:
            assert name == kernel.format(dtype)
        x = Z.double().requires_grad_()
        (x if act == NONE else torch.nn.functional.gelu(x, approximate="tanh")).sum().backward()
        ref = z * x.grad
        near(d, ref, size, K, dtype, 1.13, 2.0 ** -18 * z.abs())
        want = ref.sum(0)
        slope = 0 if act == NONE else float((2.0 ** -18 * z.abs()).norm())  # (its error: rows' are independent)
        most = 8.4e-6 if "split" in name else 3.8e-6
        assert float((sums.double() - want).norm()) <= most * float(want.norm()) + slope
        assert lib.gemm_last_device_status() == lib.GEMM_OK
    odd = torch.empty(M, N + 3, dtype=A.dtype, device="cuda")[:, 1:N + 1]
    again, sums2 = lib.gemm_fused_grad(A, B, Z, activation=GELU, bias_grad=True, out=odd)
    assert torch.equal(again, d) and torch.equal(sums, sums2)


@pytest.mark.parametrize("M,N,K", [(2304, 2560, 1600), (300, 520, 1000)])
def test_column_sums_on_streams_in_graphs_and_in_place(M, N, K):
    """Sums in parts, and the workspace of the blocks' sums, several calls at once."""
    A, B, _, Z, _ = big(M, N, K, "bf16", 0, 0)
    want, sums = lib.gemm_fused_grad(A, B, Z, activation=SILU, bias_grad=True)
    over = Z.clone()
    d, s = lib.gemm_fused_grad(A, B, over, activation=SILU, bias_grad=True, out=over)
    assert torch.equal(over, want) and torch.equal(s, sums)
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(4)]
    got = [lib.gemm_fused_grad(A, B, Z, activation=SILU, bias_grad=True, stream=side) for side in sides * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(d, want) and torch.equal(s, sums) for d, s in got)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, *lib.gemm_fused_grad(A, B, Z, activation=SILU, bias_grad=True)))
    for graph, d, s in graphs:
        d.zero_(), s.zero_()
    torch.cuda.synchronize()
    for (graph, _, _), side in zip(graphs, sides):  # side by side
        with torch.cuda.stream(side):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for _, d, s in graphs:
        assert torch.equal(d, want) and torch.equal(s, sums)
    assert lib.gemm_last_device_status() == lib.GEMM_OK


def test_rows_behind_the_last_are_left():
    for M, N, K in ((300, 520, 128), (2100, 2500, 64), (20, 4096, 2048)):
        A, B, R, Z, b = big(M, N, K, "bf16", 0, 1)
        buf = torch.full((M + 300, N + 72), 7.0, dtype=torch.bfloat16, device="cuda")
        lib.gemm_fused(A, B, bias=b, residual=R, out=buf[:M, :N])
        assert (buf[M:] == 7.0).all() and (buf[:, N:] == 7.0).all()
        lib.gemm_fused_grad(A, B, Z, activation=SILU, out=buf[:M, :N])
        assert (buf[M:] == 7.0).all() and (buf[:, N:] == 7.0).all()


def test_large_in_place_and_on_many_streams():
    """The residual read ahead of the tiles that overwrite it; several products at once."""
    M, N, K = 2304, 2560, 128
    A, B, R, Z, b = big(M, N, K, "f16", 0, 0)
    want = lib.gemm_fused(A, B, bias=b, residual=R, activation=GELU)
    dw, sw = lib.gemm_fused_grad(A, B, Z, activation=GELU, bias_grad=True)
    torch.cuda.synchronize()
    for _ in range(3):
        over, grad = R.clone(), Z.clone()
        lib.gemm_fused(A, B, bias=b, residual=over, activation=GELU, out=over)
        _, s = lib.gemm_fused_grad(A, B, grad, activation=GELU, bias_grad=True, out=grad)
        assert torch.equal(over, want) and torch.equal(grad, dw) and torch.equal(s, sw)
    sides = [torch.cuda.Stream() for _ in range(4)]
    outs = [(lib.gemm_fused(A, B, bias=b, residual=R, activation=GELU, stream=s),
             lib.gemm_fused_grad(A, B, Z, activation=GELU, bias_grad=True, stream=s)) for s in sides]
    torch.cuda.synchronize()
    for o, (d, s) in outs:
        assert torch.equal(o, want) and torch.equal(d, dw) and torch.equal(s, sw)
