"""The grouped operators' argument checks, which need no device."""
import pytest
import torch

import dense_gemm_08_gb300 as lib

FAKE = 1 << 20  # never dereferenced: the checks run before any CUDA call
BAD = lib.GEMM_ERR_INVALID_VALUE


@pytest.mark.parametrize("fn_name", ["gemm_grouped_f32", "gemm_grouped_bf16_f32acc",
                                     "gemm_grouped_f16_f32acc"])
def test_grouped_refusals(fn_name):
    good = dict(groups=4, rows=9, N=16, K=8, alpha=1.0, A=FAKE, lda=8, rows_a=9, row_index=None,
                offsets=FAKE, B=FAKE, ldb=16, stride_b=128, order_b=0, D=FAKE, ldd=16, bias=None,
                activation=0, d_type=0)
    other = {"gemm_grouped_f32": lib.GEMM_D_BF16, "gemm_grouped_bf16_f32acc": lib.GEMM_D_F16,
             "gemm_grouped_f16_f32acc": lib.GEMM_D_BF16}[fn_name]
    for change in [dict(groups=-1), dict(rows=-1), dict(N=1 << 31), dict(K=-2), dict(A=None),
                   dict(lda=7), dict(rows_a=8), dict(row_index=FAKE + 2), dict(offsets=None),
                   dict(offsets=FAKE + 2), dict(B=None), dict(ldb=15), dict(order_b=1, ldb=7),
                   dict(stride_b=-1), dict(order_b=3), dict(D=None), dict(ldd=15),
                   dict(D=FAKE + 1), dict(bias=FAKE + 1), dict(activation=7), dict(d_type=other),
                   dict(d_type=9), dict(A=FAKE + 1), dict(stride_b=(1 << 40) + 1),
                   dict(row_index=FAKE, rows_a=-1)]:
        assert getattr(lib, fn_name)(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(groups=0), dict(rows=0), dict(N=0)]:
        a = dict(good, A=None, B=None, D=None, offsets=None, **change)
        assert getattr(lib, fn_name)(**a, stream=0) == lib.GEMM_OK
    assert lib.gemm_last_kernel() == ""


@pytest.mark.parametrize("fn_name", ["gemm_grouped_wgrad_f32", "gemm_grouped_wgrad_bf16_f32acc",
                                     "gemm_grouped_wgrad_f16_f32acc"])
def test_wgrad_refusals(fn_name):
    good = dict(groups=4, rows=9, M=8, N=16, alpha=1.0, A=FAKE, lda=8, rows_a=9, row_index=None,
                offsets=FAKE, B=FAKE, ldb=16, beta=1.0, C=FAKE, ldc=16, stride_c=128, D=FAKE,
                ldd=16, stride_d=128, d_type=0)
    for change in [dict(groups=-1), dict(rows=1 << 31), dict(M=-1), dict(N=-1), dict(A=None),
                   dict(B=None), dict(lda=7), dict(ldb=15), dict(rows_a=8), dict(offsets=None),
                   dict(C=None), dict(C=FAKE + 2), dict(ldc=15), dict(stride_c=-1), dict(D=None),
                   dict(ldd=15), dict(stride_d=0), dict(d_type=5), dict(row_index=FAKE + 1)]:
        assert getattr(lib, fn_name)(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(groups=0), dict(M=0), dict(N=0)]:
        a = dict(good, A=None, B=None, C=None, D=None, offsets=None, **change)
        assert getattr(lib, fn_name)(**a, stream=0) == lib.GEMM_OK


@pytest.mark.parametrize("fn_name", ["gemm_lora_bf16_f32acc", "gemm_lora_f16_f32acc"])
def test_lora_refusals(fn_name):
    good = dict(M=5, N=16, K=8, X=FAKE, ldx=8, W=FAKE, ldw=16, order_w=0, adapters=3, rank=4,
                adapter_of_row=FAKE, scale=None, LA=FAKE, ld_a=4, stride_a=32, order_a=0, LB=FAKE,
                ld_b=16, stride_b=64, order_b=0, D=FAKE, ldd=16)
    for change in [dict(M=-1), dict(N=-1), dict(K=-1), dict(X=None), dict(ldx=7), dict(W=None),
                   dict(ldw=15), dict(order_w=2), dict(order_w=1, ldw=7), dict(adapters=-1),
                   dict(rank=-1), dict(adapter_of_row=None), dict(scale=FAKE + 2), dict(LA=None),
                   dict(ld_a=3), dict(stride_a=-1), dict(order_a=5), dict(LB=None), dict(ld_b=15),
                   dict(order_b=1, ld_b=3), dict(D=None), dict(ldd=15), dict(bias=FAKE + 2),
                   dict(activation=-1), dict(d_type=4)]:
        assert getattr(lib, fn_name)(**dict(good, **change), stream=0, check=False) == BAD, change
    for change in [dict(M=0), dict(N=0)]:
        a = dict(good, X=None, W=None, LA=None, LB=None, D=None, adapter_of_row=None, **change)
        assert getattr(lib, fn_name)(**a, stream=0) == lib.GEMM_OK


def test_group_rows_refusals():
    good = dict(rows=5, groups=3, group_of_row=FAKE, offsets=FAKE, order=FAKE, position=None)
    for change in [dict(rows=-1), dict(rows=1 << 31), dict(groups=0), dict(groups=-1),
                   dict(group_of_row=None), dict(offsets=None), dict(offsets=FAKE + 1),
                   dict(order=None), dict(position=FAKE + 3)]:
        assert lib.gemm_group_rows(**dict(good, **change), stream=0, check=False) == BAD, change


def test_stack_order():
    t = torch.zeros(3, 4, 6)
    assert lib.stack_order(t) == (lib.ROW_MAJOR, 6, 24)
    assert lib.stack_order(t.transpose(1, 2)) == (lib.COL_MAJOR, 6, 24)
    assert lib.stack_order(t[:1].expand(5, 4, 6)) == (lib.ROW_MAJOR, 6, 0)
    with pytest.raises(ValueError):
        lib.stack_order(t[:, :, ::2])
    with pytest.raises(ValueError):
        lib.stack_order(t[0])


def test_helpers_check_before_calling_the_library():
    A, B = torch.zeros(6, 8), torch.zeros(2, 8, 4)
    off = torch.zeros(3, dtype=torch.int32)
    for bad, err in [(dict(A=torch.zeros(6, 7)), ValueError), (dict(B=B.half()), TypeError),
                     (dict(offsets=off.long()), TypeError), (dict(offsets=off[:2]), ValueError),
                     (dict(row_index=off.long()), TypeError), (dict(bias=torch.zeros(4)), ValueError),
                     (dict(bias=torch.zeros(2, 4).half()), TypeError),
                     (dict(out_dtype=torch.bfloat16), TypeError),
                     (dict(out=torch.zeros(5, 4)), ValueError),
                     (dict(A=torch.zeros(8, 6).t()), ValueError),
                     (dict(A=A.int(), B=B.int()), TypeError)]:
        with pytest.raises(err):
            lib.gemm_grouped(**dict(dict(A=A, B=B, offsets=off), **bad))
    dY = torch.zeros(6, 4)
    for bad, err in [(dict(B=dY[:5]), ValueError), (dict(beta=1.0), ValueError),
                     (dict(beta=1.0, C=torch.zeros(2, 8, 4).half()), TypeError),
                     (dict(beta=1.0, C=torch.zeros(2, 8, 5)), ValueError),
                     (dict(out=torch.zeros(2, 4, 8).transpose(1, 2)), ValueError),
                     (dict(B=torch.zeros(4, 6).t()), ValueError),
                     (dict(offsets=off.float()), TypeError)]:
        with pytest.raises(err):
            lib.gemm_grouped_wgrad(**dict(dict(A=A, B=dY, offsets=off), **bad))
    h = torch.float16
    X, W = torch.zeros(6, 8, dtype=h), torch.zeros(8, 4, dtype=h)
    LA, LB = torch.zeros(3, 8, 2, dtype=h), torch.zeros(3, 2, 4, dtype=h)
    ids = torch.zeros(6, dtype=torch.int32)
    for bad, err in [(dict(X=X.float(), W=W.float()), TypeError), (dict(LB=LB[:2]), ValueError),
                     (dict(LA=LA.bfloat16()), TypeError), (dict(LA=LA[:, :7]), ValueError),
                     (dict(adapter_of_row=ids[:5]), ValueError),
                     (dict(scale=torch.zeros(2)), ValueError), (dict(bias=torch.zeros(5)), ValueError),
                     (dict(out_dtype=torch.bfloat16), TypeError),
                     (dict(W=torch.zeros(7, 4, dtype=h)), ValueError)]:
        with pytest.raises(err):
            lib.gemm_lora(**dict(dict(X=X, W=W, LA=LA, LB=LB, adapter_of_row=ids), **bad))
    with pytest.raises(TypeError):
        lib.group_rows(ids.long(), 3)
    # all well but for the device: nothing reaches the library
    for call in (lambda: lib.gemm_grouped(A, B, off), lambda: lib.gemm_grouped_wgrad(A, dY, off),
                 lambda: lib.gemm_lora(X, W, LA, LB, ids), lambda: lib.group_rows(ids, 3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
