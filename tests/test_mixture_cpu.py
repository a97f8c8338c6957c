"""Refusals of the router, the combination and the fused products, which need no device."""
import pytest
import torch

import dense_gemm_08_gb300 as lib

FAKE = 1 << 20  # never dereferenced: the checks run before any CUDA call
FAKE2 = 1 << 21
BAD = lib.GEMM_ERR_INVALID_VALUE


def test_route_refusals():
    good = dict(tokens=5, experts=16, k=4, logits=FAKE, ld=16, type=0, chosen=FAKE, weights=FAKE,
                bias=FAKE, groups=4, groups_kept=2, group_top=2)
    for change in [dict(tokens=-1), dict(tokens=1 << 31), dict(experts=0), dict(experts=1025),
                   dict(k=0), dict(k=17), dict(k=-1), dict(logits=None), dict(logits=FAKE + 2),
                   dict(ld=15), dict(type=3), dict(type=-1), dict(chosen=None),
                   dict(chosen=FAKE + 2), dict(weights=None), dict(weights=FAKE + 1),
                   dict(bias=FAKE + 2), dict(score=2), dict(renormalize=2), dict(groups=0),
                   dict(groups=3), dict(groups=33, experts=66, ld=66), dict(groups_kept=0),
                   dict(groups_kept=5), dict(group_top=0), dict(group_top=3),
                   dict(experts=64, ld=64, k=33), dict(ld=(1 << 40) + 1)]:
        assert lib.gemm_route(**dict(good, **change), stream=0, check=False) == BAD, change
    a = dict(good, tokens=0, logits=None, chosen=None, weights=None)
    assert lib.gemm_route(**a, stream=0) == lib.GEMM_OK
    assert lib.gemm_last_kernel() == ""


def test_route_grad_refusals():
    good = dict(tokens=5, experts=16, k=4, logits=FAKE, ld=16, type=1, chosen=FAKE, dweights=FAKE,
                dlogits=FAKE2, ld_d=16)
    for change in [dict(tokens=-1), dict(experts=0), dict(experts=1025), dict(k=0), dict(k=17),
                   dict(logits=None), dict(logits=FAKE + 1), dict(ld=15), dict(type=9),
                   dict(chosen=None), dict(dweights=None), dict(dweights=FAKE + 2),
                   dict(dlogits=None), dict(dlogits=FAKE + 1), dict(ld_d=15), dict(score=-1),
                   dict(renormalize=-1)]:
        assert lib.gemm_route_grad(**dict(good, **change), stream=0, check=False) == BAD, change
    a = dict(good, tokens=0, logits=None, chosen=None, dweights=None, dlogits=None)
    assert lib.gemm_route_grad(**a, stream=0) == lib.GEMM_OK


def test_combine_refusals():
    good = dict(tokens=5, k=2, N=16, Y=FAKE, ldy=16, rows_y=10, y_type=1, position=FAKE,
                weights=FAKE, residual=FAKE, ld_r=16, D=FAKE2, ldd=16, d_type=1)
    for change in [dict(tokens=-1), dict(k=-1), dict(N=-1), dict(rows_y=-1), dict(N=1 << 31),
                   dict(Y=None), dict(Y=FAKE + 1), dict(ldy=15), dict(y_type=3), dict(y_type=2),
                   dict(d_type=2), dict(position=None), dict(position=FAKE + 2),
                   dict(weights=FAKE + 2), dict(residual=FAKE + 1), dict(ld_r=15), dict(D=None),
                   dict(D=FAKE + 1), dict(ldd=15), dict(d_type=7),
                   dict(tokens=(1 << 31) - 1, k=1024)]:
        assert lib.gemm_combine(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(tokens=0), dict(N=0)]:
        a = dict(good, Y=None, position=None, weights=None, residual=None, D=None, **change)
        assert lib.gemm_combine(**a, stream=0) == lib.GEMM_OK


def test_combine_grad_refusals():
    good = dict(tokens=5, k=2, N=16, dD=FAKE, ld_d=16, d_type=0, Y=FAKE, ldy=16, rows_y=10,
                y_type=2, position=FAKE, weights=FAKE, dY=FAKE2, ld_dy=16, dweights=FAKE2)
    for change in [dict(tokens=-1), dict(k=0), dict(N=-1), dict(rows_y=-1), dict(dD=None),
                   dict(dD=FAKE + 2), dict(ld_d=15), dict(d_type=1), dict(Y=None), dict(ldy=15),
                   dict(y_type=4), dict(position=None), dict(position=FAKE + 1),
                   dict(weights=FAKE + 2), dict(dY=FAKE2 + 1), dict(ld_dy=15),
                   dict(dweights=FAKE2 + 2)]:
        assert lib.gemm_combine_grad(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(tokens=0), dict(N=0, dweights=None), dict(dY=None, dweights=None)]:
        assert lib.gemm_combine_grad(**dict(good, **change), stream=0) == lib.GEMM_OK, change


@pytest.mark.parametrize("t", ["f32", "bf16_f32acc", "f16_f32acc"])
def test_fused_refusals(t):
    good = dict(M=5, N=16, K=8, alpha=1.0, A=FAKE, lda=8, order_a=0, B=FAKE, ldb=16, order_b=0,
                D=FAKE2, ldd=16, bias=FAKE, activation=3, residual=FAKE2, ld_residual=16,
                pre=FAKE, ld_pre=16)
    fn = getattr(lib, "gemm_fused_" + t)
    for change in [dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(A=None), dict(A=FAKE + 1),
                   dict(lda=7), dict(order_a=2), dict(order_a=1, lda=4), dict(B=None),
                   dict(ldb=15), dict(order_b=1, ldb=7), dict(order_b=-1), dict(D=None),
                   dict(D=FAKE2 + 1), dict(ldd=15), dict(bias=FAKE + 2), dict(activation=4),
                   dict(activation=-1), dict(residual=FAKE + 1), dict(ld_residual=15),
                   dict(pre=FAKE + 1), dict(ld_pre=15), dict(pre=FAKE2),
                   dict(M=1 << 22, N=(1 << 21) + 1, ldb=1 << 22, ldd=1 << 22)]:
        assert fn(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(M=0), dict(N=0)]:
        a = dict(good, A=None, B=None, D=None, bias=None, residual=None, pre=None, **change)
        assert fn(**a, stream=0) == lib.GEMM_OK
    good = dict(M=5, N=16, K=8, alpha=1.0, A=FAKE, lda=8, order_a=0, B=FAKE, ldb=16, order_b=0,
                activation=2, pre=FAKE, ld_pre=16, D=FAKE2, ldd=16, dbias=FAKE2)
    fn = getattr(lib, "gemm_fused_grad_" + t)
    for change in [dict(M=-1), dict(N=-1), dict(K=1 << 31), dict(A=None), dict(lda=7),
                   dict(B=None), dict(ldb=15), dict(order_b=5), dict(D=None), dict(ldd=15),
                   dict(activation=4), dict(pre=None), dict(pre=FAKE + 1), dict(ld_pre=15),
                   dict(dbias=FAKE2 + 2)]:
        assert fn(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(M=0, dbias=None), dict(N=0)]:
        assert fn(**dict(good, A=None, B=None, D=None, pre=None, **change), stream=0) == lib.GEMM_OK


@pytest.mark.parametrize("t", ["f32", "bf16_f32acc", "f16_f32acc"])
def test_matrices_at_the_same_address(t):
    """Refused where they must not overlap, or only with the same pitch."""
    route = dict(tokens=5, experts=16, k=4, logits=FAKE, ld=16, type=1, chosen=FAKE, dweights=FAKE,
                 dlogits=FAKE, ld_d=24)
    assert lib.gemm_route_grad(**route, stream=0, check=False) == BAD
    combine = dict(tokens=5, k=2, N=16, Y=FAKE, ldy=16, rows_y=10, y_type=1, position=FAKE,
                   weights=FAKE, residual=FAKE, ld_r=16, D=FAKE2, ldd=16, d_type=1)
    for change in [dict(D=FAKE), dict(residual=FAKE2, ld_r=24)]:
        assert lib.gemm_combine(**dict(combine, **change), stream=0, check=False) == BAD, change
    grad = dict(tokens=5, k=2, N=16, dD=FAKE, ld_d=16, d_type=0, Y=2 * FAKE2, ldy=16, rows_y=10,
                y_type=2, position=FAKE, weights=FAKE, dY=FAKE2, ld_dy=16, dweights=FAKE2)
    for change in [dict(dY=FAKE), dict(dY=2 * FAKE2), dict(dweights=FAKE)]:
        assert lib.gemm_combine_grad(**dict(grad, **change), stream=0, check=False) == BAD, change
    fused = dict(M=5, N=16, K=16, alpha=1.0, A=FAKE, lda=16, order_a=0, B=2 * FAKE, ldb=16, order_b=0,
                 D=3 * FAKE, ldd=16, residual=4 * FAKE, ld_residual=16, pre=5 * FAKE, ld_pre=16)
    for change in [dict(D=FAKE), dict(D=2 * FAKE), dict(D=4 * FAKE, ldd=24), dict(pre=FAKE),
                   dict(pre=2 * FAKE), dict(pre=3 * FAKE), dict(pre=4 * FAKE)]:
        fn = getattr(lib, "gemm_fused_" + t)
        assert fn(**dict(fused, **change), stream=0, check=False) == BAD, change
    grad = dict(M=5, N=16, K=16, alpha=1.0, A=FAKE, lda=16, order_a=0, B=2 * FAKE, ldb=16, order_b=0,
                activation=2, pre=4 * FAKE, ld_pre=16, D=3 * FAKE, ldd=16, dbias=5 * FAKE)
    for change in [dict(D=FAKE), dict(D=2 * FAKE), dict(D=4 * FAKE, ldd=24), dict(dbias=FAKE),
                   dict(dbias=2 * FAKE), dict(dbias=3 * FAKE), dict(dbias=4 * FAKE)]:
        fn = getattr(lib, "gemm_fused_grad_" + t)
        assert fn(**dict(grad, **change), stream=0, check=False) == BAD, change


def test_silu_is_of_the_fused_products_only():
    assert lib.gemm_bf16_f32acc_ex(8, 8, 8, 1.0, FAKE, 8, 0, FAKE, 8, 0, 0.0, None, 8, FAKE2, 8, 0,
                                   activation=lib.GEMM_ACT_SILU, stream=0, check=False) == BAD


def test_helpers_check_before_calling_the_library():
    x = torch.zeros(6, 8)
    ids, w = torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 2)
    for bad, err in [(dict(logits=x.int()), TypeError), (dict(logits=x[0]), ValueError),
                     (dict(logits=x.t()), ValueError), (dict(logits=x[:, ::2]), ValueError),
                     (dict(bias=torch.zeros(7)), ValueError), (dict(bias=x[0].half()), TypeError)]:
        with pytest.raises(err):
            lib.route(**dict(dict(logits=x, k=2), **bad))
    for bad, err in [(dict(chosen=ids.long()), TypeError), (dict(chosen=ids[:5]), ValueError),
                     (dict(dweights=w.half()), TypeError), (dict(dweights=w[:, :1]), ValueError),
                     (dict(out=x.half()), TypeError), (dict(out=x[:5]), ValueError),
                     (dict(logits=x.double()), TypeError)]:
        with pytest.raises(err):
            lib.route_grad(**dict(dict(logits=x, chosen=ids, dweights=w), **bad))
    Y = torch.zeros(12, 8, dtype=torch.bfloat16)
    for bad, err in [(dict(Y=Y.int()), TypeError), (dict(position=ids.long()), TypeError),
                     (dict(position=ids.t()), ValueError), (dict(weights=w[:5]), ValueError),
                     (dict(weights=w.half()), TypeError), (dict(residual=x), TypeError),
                     (dict(residual=Y[:5]), ValueError), (dict(out=x.half()), TypeError),
                     (dict(out=x, out_dtype=torch.bfloat16), TypeError),
                     (dict(out_dtype=torch.float16), TypeError), (dict(Y=Y.t()), ValueError)]:
        with pytest.raises(err):
            lib.combine(**dict(dict(Y=Y, position=ids, weights=w), **bad))
    for bad, err in [(dict(dD=x.half()), TypeError), (dict(dD=x[:5]), ValueError),
                     (dict(out=Y.float()), TypeError), (dict(out=Y[:5]), ValueError),
                     (dict(position=ids[0]), ValueError), (dict(weights=w.double()), TypeError)]:
        with pytest.raises(err):
            lib.combine_grad(**dict(dict(dD=x, Y=Y, position=ids, weights=w), **bad))
    A, B, R = torch.zeros(6, 8), torch.zeros(8, 4), torch.zeros(6, 4)
    for bad, err in [(dict(A=A.half()), TypeError), (dict(B=B[:7]), ValueError),
                     (dict(bias=torch.zeros(5)), ValueError), (dict(residual=R.half()), TypeError),
                     (dict(residual=R[:5]), ValueError), (dict(out=R.half()), TypeError),
                     (dict(out=torch.zeros(4, 6).t()), ValueError),
                     (dict(A=A.int(), B=B.int()), TypeError),
                     (dict(A=torch.zeros(6, 16)[:, ::2]), ValueError)]:
        with pytest.raises(err):
            lib.gemm_fused(**dict(dict(A=A, B=B), **bad))
    for bad, err in [(dict(pre=None, activation=lib.GEMM_ACT_GELU), ValueError),
                     (dict(pre=R.half()), TypeError), (dict(pre=R[:, :3]), ValueError),
                     (dict(out=R[:5]), ValueError)]:
        with pytest.raises(err):
            lib.gemm_fused_grad(**dict(dict(A=A, B=B, pre=R), **bad))
    # all well but for the device: nothing reaches the library
    for call in (lambda: lib.route(x, 2), lambda: lib.route_grad(x, ids, w),
                 lambda: lib.combine(Y, ids, w), lambda: lib.combine_grad(x, Y, ids, w),
                 lambda: lib.gemm_fused(A, B), lambda: lib.gemm_fused_grad(A, B, R)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
