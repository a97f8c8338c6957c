"""The combination of experts' rows and its gradients against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import TORCH, f64
from mixture_harness import HALF_STEP, check, rounding, stored

pytestmark = pytest.mark.gpu


def make(T, k, N, y, d, rows=None, extra=0, seed=0, weights=True, residual=True):
    rng = np.random.default_rng([T, k, N, seed])
    rows = T * k if rows is None else rows
    Y = stored(rng.standard_normal((rows, N)), y, extra)
    at = np.full(T * k, -1, dtype=np.int32)
    n = min(rows, T * k)
    at[rng.permutation(T * k)[:n]] = rng.permutation(rows)[:n]
    at = torch.from_numpy(at.reshape(T, k)).cuda()
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32)).cuda() if weights else None
    R = stored(rng.standard_normal((T, N)), d, extra) if residual else None
    return Y, at, w, R


def reference(Y, at, w, R):
    """(D, sum of the terms' magnitudes)"""
    y, p = f64(Y), at.cpu().numpy()
    T, k = p.shape
    d, size = np.zeros((T, y.shape[1])), np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= p[t, j] < y.shape[0]:
                v = y[p[t, j]] * (1.0 if w is None else float(w[t, j]))
                d[t] += v
                size[t] += np.abs(v)
    if R is not None:
        d += f64(R)
        size += np.abs(f64(R))
    return d, size


def tolerance(size, k, out, ref):
    """k + 1 additions and as many products, each half a step of FP32 of at most `size`."""
    return size * (2 * k + 2) * 2.0 ** -24 + rounding(out, ref)


SIZES = [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (5, 8, 33), (17, 4, 64), (64, 3, 130), (9, 11, 257),
         (2, 32, 1000), (40, 1, 8), (33, 8, 2049)]


@pytest.mark.parametrize("y,d", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                 ("f16", "f32")])
@pytest.mark.parametrize("T,k,N", SIZES)
@pytest.mark.parametrize("extra", [0, 3, 8])
def test_combine(y, d, T, k, N, extra):
    for weights, residual in ((True, True), (False, False)):
        Y, at, w, R = make(T, k, N, y, d, extra=extra, weights=weights, residual=residual)
        ref, size = reference(Y, at, w, R)
        tol = tolerance(size, k, d, ref)
        got = lib.combine(Y, at, weights=w, residual=R, out_dtype=TORCH[d])
        assert lib.gemm_last_kernel() == "combine"
        check(got, ref, tol)
        out = stored(np.zeros((T, N)), d, 5, fill=7.0)
        assert torch.equal(lib.combine(Y, at, weights=w, residual=R, out=out), got)
        assert (out.as_strided((T, 5), out.stride(), out.storage_offset() + N)[:T] == 7.0).all()
        if residual:  # in place
            over = R.clone()
            assert torch.equal(lib.combine(Y, at, weights=w, residual=over, out=over), got)


@pytest.mark.parametrize("y,d", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                 ("f16", "f32")])
@pytest.mark.parametrize("T,k,N", SIZES)
@pytest.mark.parametrize("extra", [0, 3, 8])
def test_gradients(y, d, T, k, N, extra):
    for weights in (True, False):
        Y, at, w, _ = make(T, k, N, y, d, rows=max(T * k - T // 2, 1), extra=extra, weights=weights)
        rng = np.random.default_rng(N)
        dD = stored(rng.standard_normal((T, N)), d, extra)
        g, yv, p = f64(dD), f64(Y), at.cpu().numpy()
        rows = yv.shape[0]
        want, tol = np.full((rows, N), 7.0), np.zeros((rows, N))
        dw, dtol = np.zeros((T, k)), np.zeros((T, k))
        for t in range(T):
            for j in range(k):
                r = p[t, j]
                if not 0 <= r < rows:
                    continue
                want[r] = g[t] * (1.0 if w is None else float(w[t, j]))
                tol[r] = rounding(y, want[r]) + 2.0 ** -23 * np.abs(want[r])
                dw[t, j] = g[t] @ yv[r]
                # N products summed: a thread's share (at most N / 32 of them, or 8), 5 shuffles, 8 warps
                dtol[t, j] = (np.abs(g[t]) @ np.abs(yv[r])) * (N / 32 + 8 + 16) * 2.0 ** -24
        out = stored(np.full((rows, N), 7.0), y, extra, fill=9.0)
        dY, got = lib.combine_grad(dD, Y, at, weights=w, out=out)
        assert lib.gemm_last_kernel() == "combine_grad" and dY is out
        check(dY, want, tol, "dY")
        check(got, dw, dtol + 1e-30, "dweights")
        again, none = lib.combine_grad(dD, Y, at, weights=w, weight_grad=False)
        assert none is None
        named = torch.zeros(rows, dtype=torch.bool)
        named[[r for r in p.ravel() if 0 <= r < rows]] = True
        assert torch.equal(again.cpu()[named], dY.cpu()[named])


def test_the_gather_and_its_gradient():
    """combine without weights is the gradient of a gather: <gather(x), g> = <x, combine(g)>."""
    T, k, N = 50, 4, 96
    ids = torch.randint(0, 8, (T * k,), device="cuda", dtype=torch.int32)
    ids[::7] = -1
    offsets, order, position = lib.group_rows(ids, 8)
    rows = int(offsets[-1])
    x, g = torch.randn(T, N, device="cuda"), torch.randn(T * k, N, device="cuda")
    gathered = x.double()[(order[:rows] // k).long()]
    back = lib.combine(g[:rows], position.view(T, k))
    a, b = (gathered * g[:rows].double()).sum(), (x.double() * back.double()).sum()
    # back's sums: k additions of 2^-24 each
    assert abs(a - b) <= (x.abs().double() * back.abs().double() + 4).sum() * 2.0 ** -22


def test_gradients_against_differences():
    """combine is linear in Y and in the weights: differences of any step are exact but for rounding."""
    T, k, N = 6, 3, 40
    Y, at, w, _ = make(T, k, N, "f32", "f32", residual=False)
    g = torch.randn(T, N, device="cuda")
    dY, dw = lib.combine_grad(g, Y, at, weights=w)

    def value(y, u):
        return (reference(y, at, u, None)[0] * f64(g)).sum()

    base = value(Y, w)
    rng = np.random.default_rng(0)
    for _ in range(6):
        r, c = rng.integers(T * k), rng.integers(N)
        up = Y.double().clone()
        up[r, c] += 1.0
        assert abs(value(up, w) - base - float(dY[r, c])) < 1e-5 * (1 + abs(float(dY[r, c])))
        t, j = rng.integers(T), rng.integers(k)
        uw = w.double().clone()
        uw[t, j] += 1.0
        assert abs(value(Y, uw) - base - float(dw[t, j])) < 1e-5 * (1 + abs(float(dw[t, j])))


def test_rows_without_a_place_and_special_values():
    T, k, N = 5, 3, 24
    Y, at, w, R = make(T, k, N, "bf16", "bf16")
    clean = lib.combine(Y, at, weights=w, residual=R)
    # an infinity and a NaN in rows reach the tokens that have them, in places out of range nothing does
    p = at.clone()
    p[1] = torch.tensor([-1, T * k, 1 << 30], dtype=torch.int32)
    w2 = w.clone()
    w2[1] = float("nan")
    got = lib.combine(Y, p, weights=w2, residual=R)
    assert torch.equal(got[1], R[1])
    Y2 = Y.clone()
    Y2[int(at[2, 0]), 5] = float("nan")
    Y2[int(at[3, 1]), 6] = float("inf")
    got = lib.combine(Y2, at, weights=w, residual=R)
    hit = torch.zeros(T, N, dtype=torch.bool)
    hit[2, 5] = hit[3, 6] = True
    assert torch.isnan(got[2, 5]) and torch.isinf(got[3, 6])
    assert torch.equal(got.cpu()[~hit], clean.cpu()[~hit])
    # no choices at all: the residual, or zeros; no rows of Y at all
    none = torch.zeros(T, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(lib.combine(Y, none, residual=R), R)
    assert (lib.combine(Y, none) == 0).all()
    assert torch.equal(lib.combine(Y[:0], at, weights=w, residual=R), R)
    dY, dw = lib.combine_grad(R, Y[:0], at, weights=w)
    assert dY.shape == (0, N) and (dw == 0).all()


def test_streams_and_graphs():
    T, k, N = 200, 4, 512
    Y, at, w, R = make(T, k, N, "f16", "f16")
    want = lib.combine(Y, at, weights=w, residual=R)
    dY, dw = lib.combine_grad(R, Y, at, weights=w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib.combine(Y, at, weights=w, residual=R, stream=s)
    gY, gw = lib.combine_grad(R, Y, at, weights=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(gY, dY) and torch.equal(gw, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.combine(Y, at, weights=w, residual=R)
        oY, ow = lib.combine_grad(out, Y, at, weights=w)
    graph.replay()
    assert torch.equal(out, want)
    eY, ew = lib.combine_grad(want, Y, at, weights=w)
    assert torch.equal(oY, eY) and torch.equal(ow, ew)


def test_offsets_past_32_bits():
    """Rows of Y, D and dY more than 2^31 elements apart."""
    T, k, N = 2, 2, 40
    pitch = (1 << 30) + 8
    Y, at, w, R = make(T, k, N, "bf16", "bf16")
    far = torch.empty(3 * pitch + N, dtype=torch.bfloat16, device="cuda").as_strided((4, N), (pitch, 1))
    far.copy_(Y)
    want = lib.combine(Y, at, weights=w, residual=R)
    assert torch.equal(lib.combine(far, at, weights=w, residual=R), want)
    dY, dw = lib.combine_grad(R, Y, at, weights=w)
    gY, gw = lib.combine_grad(R, far, at, weights=w, out=torch.empty_like(Y))
    assert torch.equal(gY, dY) and torch.equal(gw, dw)
    lib.combine_grad(R, Y, at, weights=w, out=far)
    assert torch.equal(far.contiguous(), dY)
    lib.combine(Y, at, weights=w, residual=R, out=far[:3:2])
    assert torch.equal(far[:3:2].contiguous(), want)


@pytest.mark.parametrize("T,k,N", [(70000, 1, 8), (4097, 8, 1024)])
def test_many_tokens(T, k, N):
    Y = torch.randn(T * k, N, device="cuda").bfloat16()
    at = torch.randperm(T * k, device="cuda").to(torch.int32).view(T, k)
    w = torch.rand(T, k, device="cuda")
    ref = (Y.double()[at.long()] * w.double()[..., None]).sum(1)
    got = lib.combine(Y, at, weights=w, out_dtype=torch.float32).double()
    size = (Y.double().abs()[at.long()] * w.double()[..., None]).sum(1)
    assert ((got - ref).abs() <= size * (2 * k + 2) * 2.0 ** -24).all()
    dD = torch.randn(T, N, device="cuda")
    dY, dw = lib.combine_grad(dD, Y, at, weights=w)
    want = (dD.double()[:, None] * w.double()[..., None]).view(T * k, N)
    assert ((dY[at.view(-1).long()].double() - want).abs() <= want.abs() * (HALF_STEP["bf16"] * 1.001) +
            1e-38).all()
    ref = (dD.double()[:, None] * Y.double()[at.long()]).sum(-1)
    size = (dD.double().abs()[:, None] * Y.double().abs()[at.long()]).sum(-1)
    assert ((dw.double() - ref).abs() <= size * (N / 32 + 24) * 2.0 ** -24).all()


@pytest.mark.parametrize("y,d", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                 ("f16", "f32")])
@pytest.mark.parametrize("T,k,N", [(3400, 1, 8192), (1701, 2, 9001), (3300, 3, 2575), (900, 5, 8200), (1777, 8, 2100),
                                   (1640, 11, 2055), (700, 20, 2080), (7001, 2, 2049), (701, 8, 1056), (1500, 4, 515),
                                   (4500, 2, 1032), (6000, 2, 900), (5000, 1, 8200), (3001, 4, 777)])
def test_large_batches(y, d, T, k, N):
    """Rows by bulk copy: several runs of columns, sets of rows, odd ends, rows without a place."""
    g = torch.Generator(device="cuda").manual_seed(T)
    t, u = TORCH[y], TORCH[d]
    ld = -(-N // 8) * 8

    def normal(r, kind):
        return torch.empty(r, ld, device="cuda", dtype=kind).normal_(generator=g)[:, :N]

    Y, R = normal(T * k, t), normal(T, u)
    at = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32)
    at[::7] = -1
    at[3::50] = T * k + 5
    at = at.view(T, k)
    inside = (at >= 0) & (at < T * k)
    w = torch.rand(T, k, generator=g, device="cuda")
    w[~inside] = float("nan")
    rows = Y.double()[at.long().clamp(0, T * k - 1)] * inside[..., None]
    wd = torch.where(inside, w, torch.zeros_like(w)).double()
    for weights, residual in ((w, R), (None, None)):
        s = wd if weights is not None else inside.double()
        ref, size = (rows * s[..., None]).sum(1), (rows.abs() * s[..., None]).sum(1)
        if residual is not None:
            ref, size = ref + R.double(), size + R.double().abs()
        tol = size * (2 * k + 2) * 2.0 ** -24 + ref.abs() * HALF_STEP[d] * 1.001 + 2.0 ** -24
        out = torch.full((T, ld + 8), 7.0, device="cuda", dtype=u)
        got = lib.combine(Y, at, weights=weights, residual=residual, out=out[:, :N])
        row = N * Y.element_size()
        bulk = row >= 2048 and row * k >= 8192 and row * k * T >= 32 << 20
        assert lib.gemm_last_kernel() == ("combine<bulk>" if bulk else "combine")
        assert ((got.double() - ref).abs() <= tol).all() and (out[:, N:] == 7.0).all()
        odd = torch.empty(T, N + 1, device="cuda", dtype=u)[:, 1:]  # rows off 16 bytes
        assert torch.equal(lib.combine(Y, at, weights=weights, residual=residual, out=odd), got)
        if residual is not None:
            over = R.clone()
            assert torch.equal(lib.combine(Y, at, weights=w, residual=over, out=over), got)
    dD = normal(T, u)
    for weights in (w, None):
        s = wd if weights is not None else inside.double()
        buf = torch.full((T * k, ld), 7.0, device="cuda", dtype=t)
        dY, dw = lib.combine_grad(dD, Y, at, weights=weights, out=buf[:, :N])
        row = N * Y.element_size()
        bulk = row >= 1280 and row * k >= 4096 and row * k * T >= 16 << 20
        bulk = bulk and (k > 1 or (row >= 8192 and row * T >= 64 << 20))
        assert lib.gemm_last_kernel() == ("combine_grad<bulk>" if bulk else "combine_grad")
        want = torch.full((T * k, N), 7.0, device="cuda", dtype=torch.float64)
        want[at[inside].long()] = (dD.double()[:, None] * s[..., None])[inside]
        assert ((dY.double() - want).abs() <= want.abs() * HALF_STEP[y] * 1.001 + 2.0 ** -24).all()
        assert (buf[:, N:] == 7.0).all()
        ref = (dD.double()[:, None] * rows).sum(-1)
        size = (dD.double().abs()[:, None] * rows.abs()).sum(-1)
        # (a thread's share: at most N / 32 products and 8, then 5 shuffles and 8 warps)
        assert ((dw.double() - ref).abs() <= size * (N / 32 + 8 + 16) * 2.0 ** -24).all()
        only, none = lib.combine_grad(dD, Y, at, weights=weights, weight_grad=False)
        assert none is None and torch.equal(only[at[inside].long()], dY[at[inside].long()])
    assert lib.gemm_last_device_status() == lib.GEMM_OK


def test_large_batches_on_streams_and_in_graphs():
    T, k, N = 3200, 4, 2048
    Y, at, w, R = make(T, k, N, "bf16", "bf16")
    want = lib.combine(Y, at, weights=w, residual=R)
    assert lib.gemm_last_kernel() == "combine<bulk>"
    dY, dw = lib.combine_grad(R, Y, at, weights=w)
    assert lib.gemm_last_kernel() == "combine_grad<bulk>"
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [(lib.combine(Y, at, weights=w, residual=R, stream=s),
            *lib.combine_grad(R, Y, at, weights=w, stream=s)) for s in sides]
    torch.cuda.synchronize()
    for a, b, c in got:
        assert torch.equal(a, want) and torch.equal(b, dY) and torch.equal(c, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.combine(Y, at, weights=w, residual=R)
        oY, ow = lib.combine_grad(R, Y, at, weights=w)
    graph.replay()
    assert torch.equal(out, want) and torch.equal(oY, dY) and torch.equal(ow, dw)
