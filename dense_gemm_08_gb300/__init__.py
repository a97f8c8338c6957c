"""Python binding of the GB300 GEMM library's C ABI (include/gemm.h and
include/gemm_probe.h).

Argument marshalling only: every function here forwards to the in-tree
CUDA library ``libdense_gemm_08_gb300.so``; all arithmetic runs in its
kernels.  Importing this package without the built library raises at the
first call (there is no CPU fallback).

Same names as the C ABI:
    gemm_f32, gemm_bf16_f32acc, gemm_f16_f32acc, gemm_bf16_f32acc_ex,
    gemm_f32_noalloc, gemm_status_string, gemm_last_device_status, gemm_last_kernel,
    gemm_memory_info, gemm_release_memory,
    gemm_group_rows,
    gemm_grouped_f32, gemm_grouped_bf16_f32acc, gemm_grouped_f16_f32acc,
    gemm_grouped_wgrad_f32, gemm_grouped_wgrad_bf16_f32acc, gemm_grouped_wgrad_f16_f32acc,
    gemm_lora_bf16_f32acc, gemm_lora_f16_f32acc,
    gemm_probe_tc_bf16, gemm_probe_fma_f32, gemm_probe_wait_timeout
Pointer arguments take an integer device address or a torch CUDA tensor;
``stream`` takes an integer ``cudaStream_t``, a ``torch.cuda.Stream`` or None
(torch's current stream).  A non-zero status raises ``GemmError``.

``gemm(...)`` is a convenience wrapper for torch tensors that reads each
operand's storage order and leading dimension from its strides; so are
``group_rows(...)``, ``gemm_grouped(...)``, ``gemm_grouped_wgrad(...)`` and
``gemm_lora(...)`` for the grouped operators.
"""
from __future__ import annotations

import ctypes
import os
import threading

ROW_MAJOR = 0
COL_MAJOR = 1

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = 1
GEMM_ERR_UNSUPPORTED_DEVICE = 2
GEMM_ERR_LAUNCH = 3
GEMM_ERR_TIMEOUT = 4
GEMM_ERR_INTERNAL = 5

# DENSE_GEMM_08_GB300_LIB names another build of the same library (for
# example a variant from _build.build_variant); by default the in-tree build.
LIB_PATH = os.environ.get("DENSE_GEMM_08_GB300_LIB") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "libdense_gemm_08_gb300.so")
EXPORTED = ("gemm_f32", "gemm_bf16_f32acc", "gemm_f16_f32acc", "gemm_bf16_f32acc_ex",
            "gemm_f32_noalloc", "gemm_status_string", "gemm_last_device_status",
            "gemm_last_kernel", "gemm_memory_info", "gemm_release_memory",
            "gemm_group_rows", "gemm_grouped_f32", "gemm_grouped_bf16_f32acc",
            "gemm_grouped_f16_f32acc", "gemm_grouped_wgrad_f32",
            "gemm_grouped_wgrad_bf16_f32acc", "gemm_grouped_wgrad_f16_f32acc",
            "gemm_lora_bf16_f32acc", "gemm_lora_f16_f32acc",
            "gemm_probe_tc_bf16", "gemm_probe_fma_f32", "gemm_probe_wait_timeout")

GEMM_ACT_NONE = 0
GEMM_ACT_RELU = 1
GEMM_ACT_GELU = 2
GEMM_D_F32 = 0
GEMM_D_BF16 = 1
GEMM_D_F16 = 2  # the grouped operators with FP16 inputs only


class MemoryInfo(ctypes.Structure):
    """gemm_memory_info_t: what the library holds on the current device."""
    _fields_ = [("split_streams", ctypes.c_uint64), ("split_bytes", ctypes.c_uint64),
                ("pool_used_bytes", ctypes.c_uint64), ("pool_reserved_bytes", ctypes.c_uint64)]


class Epilogue(ctypes.Structure):
    """gemm_epilogue_t: bias (device pointer or None), activation, d_type."""
    _fields_ = [("bias", ctypes.c_void_p), ("activation", ctypes.c_int), ("d_type", ctypes.c_int)]

_lock = threading.Lock()
_lib = None


class GemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({gemm_status_string(status)})")
        self.status = status


def library() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"CUDA library {LIB_PATH} is not built; run __graft_entry__.build() "
                    "(or python dense_gemm_08_gb300/_build.py)")
            lib = ctypes.CDLL(LIB_PATH)
            i64, f32, vp, ip = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
            sig = [i64, i64, i64, f32, vp, i64, ip, vp, i64, ip, f32, vp, i64, vp, i64, ip, vp]
            lib.gemm_f32.argtypes = sig
            lib.gemm_f32.restype = ip
            lib.gemm_bf16_f32acc.argtypes = sig
            lib.gemm_bf16_f32acc.restype = ip
            lib.gemm_f16_f32acc.argtypes = sig
            lib.gemm_f16_f32acc.restype = ip
            lib.gemm_bf16_f32acc_ex.argtypes = sig[:-1] + [ctypes.POINTER(Epilogue), vp]
            lib.gemm_bf16_f32acc_ex.restype = ip
            lib.gemm_f32_noalloc.argtypes = sig
            lib.gemm_f32_noalloc.restype = ip
            lib.gemm_status_string.argtypes = [ip]
            lib.gemm_status_string.restype = ctypes.c_char_p
            lib.gemm_last_device_status.argtypes = [vp]
            lib.gemm_last_device_status.restype = ip
            lib.gemm_last_kernel.argtypes = []
            lib.gemm_last_kernel.restype = ctypes.c_char_p
            lib.gemm_memory_info.argtypes = [ctypes.POINTER(MemoryInfo)]
            lib.gemm_memory_info.restype = ip
            lib.gemm_release_memory.argtypes = []
            lib.gemm_release_memory.restype = ip
            ep = ctypes.POINTER(Epilogue)
            lib.gemm_group_rows.argtypes = [i64, i64, vp, vp, vp, vp, vp]
            lib.gemm_group_rows.restype = ip
            for t in ("f32", "bf16_f32acc", "f16_f32acc"):
                fn = getattr(lib, "gemm_grouped_" + t)
                fn.argtypes = [i64, i64, i64, i64, f32, vp, i64, i64, vp, vp, vp, i64, i64, ip,
                               vp, i64, ep, vp]
                fn.restype = ip
                fn = getattr(lib, "gemm_grouped_wgrad_" + t)
                fn.argtypes = [i64, i64, i64, i64, f32, vp, i64, i64, vp, vp, vp, i64, f32, vp,
                               i64, i64, vp, i64, i64, ip, vp]
                fn.restype = ip
            for t in ("bf16_f32acc", "f16_f32acc"):
                fn = getattr(lib, "gemm_lora_" + t)
                fn.argtypes = [i64, i64, i64, vp, i64, vp, i64, ip, i64, i64, vp, vp, vp, i64,
                               i64, ip, vp, i64, i64, ip, vp, i64, ep, vp]
                fn.restype = ip
            dp = ctypes.POINTER(ctypes.c_double)
            lib.gemm_probe_tc_bf16.argtypes = [ip, i64, dp, vp]
            lib.gemm_probe_tc_bf16.restype = ip
            lib.gemm_probe_fma_f32.argtypes = [i64, dp, vp]
            lib.gemm_probe_fma_f32.restype = ip
            lib.gemm_probe_wait_timeout.argtypes = [ctypes.c_uint64, vp]
            lib.gemm_probe_wait_timeout.restype = ip
            _lib = lib
    return _lib


def _addr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()  # torch tensor


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream  # torch.cuda.Stream


def _call(fn_name, M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd,
          order_cd, stream, check):
    fn = getattr(library(), fn_name)
    st = fn(int(M), int(N), int(K), float(alpha), _addr(A), int(lda), int(order_a), _addr(B),
            int(ldb), int(order_b), float(beta), _addr(C), int(ldc), _addr(D), int(ldd),
            int(order_cd), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, fn_name)
    return st


def gemm_f32(M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd, order_cd,
             stream=None, check=True) -> int:
    """FP32 GEMM on the CUDA cores (see include/gemm.h)."""
    return _call("gemm_f32", M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D,
                 ldd, order_cd, stream, check)


def gemm_bf16_f32acc(M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd,
                     order_cd, stream=None, check=True) -> int:
    """BF16-input, FP32-accumulate GEMM (tensor cores when TMA applies; see include/gemm.h)."""
    return _call("gemm_bf16_f32acc", M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C,
                 ldc, D, ldd, order_cd, stream, check)


def gemm_f16_f32acc(M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd,
                    order_cd, stream=None, check=True) -> int:
    """FP16-input, FP32-accumulate GEMM (same kernels as gemm_bf16_f32acc)."""
    return _call("gemm_f16_f32acc", M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C,
                 ldc, D, ldd, order_cd, stream, check)


def gemm_bf16_f32acc_ex(M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd,
                        order_cd, bias=None, activation=GEMM_ACT_NONE, d_type=GEMM_D_F32,
                        stream=None, check=True) -> int:
    """gemm_bf16_f32acc with a fused epilogue: D = act(alpha*AB + beta*C + bias), FP32 or BF16."""
    ep = Epilogue(_addr(bias), int(activation), int(d_type))
    st = library().gemm_bf16_f32acc_ex(
        int(M), int(N), int(K), float(alpha), _addr(A), int(lda), int(order_a), _addr(B),
        int(ldb), int(order_b), float(beta), _addr(C), int(ldc), _addr(D), int(ldd),
        int(order_cd), ctypes.byref(ep), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_bf16_f32acc_ex")
    return st


def gemm_f32_noalloc(M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C, ldc, D, ldd,
                     order_cd, stream=None, check=True) -> int:
    """gemm_f32 that allocates nothing: its split-K scratch is a fixed 32 MiB
    array inside the library (for callers that cannot allocate device memory;
    see include/gemm.h for the limits)."""
    return _call("gemm_f32_noalloc", M, N, K, alpha, A, lda, order_a, B, ldb, order_b, beta, C,
                 ldc, D, ldd, order_cd, stream, check)


def gemm_status_string(status: int) -> str:
    return library().gemm_status_string(int(status)).decode()


def gemm_last_device_status(stream=None) -> int:
    return int(library().gemm_last_device_status(_stream(stream)))


def gemm_last_kernel() -> str:
    return library().gemm_last_kernel().decode()


def gemm_memory_info(check=True) -> dict:
    """What the library holds on the current device between calls (see include/gemm.h)."""
    info = MemoryInfo()
    st = library().gemm_memory_info(ctypes.byref(info))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_memory_info")
    return {name: int(getattr(info, name)) for name, _ in MemoryInfo._fields_}


def gemm_release_memory(check=True) -> int:
    """Synchronise the device, free every stream's split counters and trim the pool."""
    st = int(library().gemm_release_memory())
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_release_memory")
    return st


def gemm_group_rows(rows, groups, group_of_row, offsets, order, position=None, stream=None,
                    check=True) -> int:
    """Rows grouped by a number: offsets, order and (optional) positions (see include/gemm.h)."""
    st = library().gemm_group_rows(int(rows), int(groups), _addr(group_of_row), _addr(offsets),
                                   _addr(order), _addr(position), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_group_rows")
    return st


def _call_grouped(fn_name, groups, rows, N, K, alpha, A, lda, rows_a, row_index, offsets, B, ldb,
                  stride_b, order_b, D, ldd, bias, activation, d_type, stream, check):
    ep = Epilogue(_addr(bias), int(activation), int(d_type))
    st = getattr(library(), fn_name)(
        int(groups), int(rows), int(N), int(K), float(alpha), _addr(A), int(lda), int(rows_a),
        _addr(row_index), _addr(offsets), _addr(B), int(ldb), int(stride_b), int(order_b),
        _addr(D), int(ldd), ctypes.byref(ep), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, fn_name)
    return st


def gemm_grouped_f32(groups, rows, N, K, alpha, A, lda, rows_a, row_index, offsets, B, ldb,
                     stride_b, order_b, D, ldd, bias=None, activation=GEMM_ACT_NONE,
                     d_type=GEMM_D_F32, stream=None, check=True) -> int:
    """D(r, :) = act(alpha * A(idx(r), :) B_g + bias_g), FP32 on the CUDA cores."""
    return _call_grouped("gemm_grouped_f32", groups, rows, N, K, alpha, A, lda, rows_a, row_index,
                         offsets, B, ldb, stride_b, order_b, D, ldd, bias, activation, d_type,
                         stream, check)


def gemm_grouped_bf16_f32acc(groups, rows, N, K, alpha, A, lda, rows_a, row_index, offsets, B,
                             ldb, stride_b, order_b, D, ldd, bias=None,
                             activation=GEMM_ACT_NONE, d_type=GEMM_D_F32, stream=None,
                             check=True) -> int:
    """D(r, :) = act(alpha * A(idx(r), :) B_g + bias_g), BF16 inputs, FP32 or BF16 D."""
    return _call_grouped("gemm_grouped_bf16_f32acc", groups, rows, N, K, alpha, A, lda, rows_a,
                         row_index, offsets, B, ldb, stride_b, order_b, D, ldd, bias, activation,
                         d_type, stream, check)


def gemm_grouped_f16_f32acc(groups, rows, N, K, alpha, A, lda, rows_a, row_index, offsets, B, ldb,
                            stride_b, order_b, D, ldd, bias=None, activation=GEMM_ACT_NONE,
                            d_type=GEMM_D_F32, stream=None, check=True) -> int:
    """D(r, :) = act(alpha * A(idx(r), :) B_g + bias_g), FP16 inputs, FP32 or FP16 D."""
    return _call_grouped("gemm_grouped_f16_f32acc", groups, rows, N, K, alpha, A, lda, rows_a,
                         row_index, offsets, B, ldb, stride_b, order_b, D, ldd, bias, activation,
                         d_type, stream, check)


def _call_wgrad(fn_name, groups, rows, M, N, alpha, A, lda, rows_a, row_index, offsets, B, ldb,
                beta, C, ldc, stride_c, D, ldd, stride_d, d_type, stream, check):
    st = getattr(library(), fn_name)(
        int(groups), int(rows), int(M), int(N), float(alpha), _addr(A), int(lda), int(rows_a),
        _addr(row_index), _addr(offsets), _addr(B), int(ldb), float(beta), _addr(C), int(ldc),
        int(stride_c), _addr(D), int(ldd), int(stride_d), int(d_type), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, fn_name)
    return st


def gemm_grouped_wgrad_f32(groups, rows, M, N, alpha, A, lda, rows_a, row_index, offsets, B, ldb,
                           beta, C, ldc, stride_c, D, ldd, stride_d, d_type=GEMM_D_F32,
                           stream=None, check=True) -> int:
    """D_g = alpha * A_g^T B_g + beta * C_g over each group's rows, FP32 on the CUDA cores."""
    return _call_wgrad("gemm_grouped_wgrad_f32", groups, rows, M, N, alpha, A, lda, rows_a,
                       row_index, offsets, B, ldb, beta, C, ldc, stride_c, D, ldd, stride_d,
                       d_type, stream, check)


def gemm_grouped_wgrad_bf16_f32acc(groups, rows, M, N, alpha, A, lda, rows_a, row_index, offsets,
                                   B, ldb, beta, C, ldc, stride_c, D, ldd, stride_d,
                                   d_type=GEMM_D_F32, stream=None, check=True) -> int:
    """D_g = alpha * A_g^T B_g + beta * C_g over each group's rows, BF16 inputs."""
    return _call_wgrad("gemm_grouped_wgrad_bf16_f32acc", groups, rows, M, N, alpha, A, lda, rows_a,
                       row_index, offsets, B, ldb, beta, C, ldc, stride_c, D, ldd, stride_d,
                       d_type, stream, check)


def gemm_grouped_wgrad_f16_f32acc(groups, rows, M, N, alpha, A, lda, rows_a, row_index, offsets, B,
                                  ldb, beta, C, ldc, stride_c, D, ldd, stride_d,
                                  d_type=GEMM_D_F32, stream=None, check=True) -> int:
    """D_g = alpha * A_g^T B_g + beta * C_g over each group's rows, FP16 inputs."""
    return _call_wgrad("gemm_grouped_wgrad_f16_f32acc", groups, rows, M, N, alpha, A, lda, rows_a,
                       row_index, offsets, B, ldb, beta, C, ldc, stride_c, D, ldd, stride_d,
                       d_type, stream, check)


def _call_lora(fn_name, M, N, K, X, ldx, W, ldw, order_w, adapters, rank, adapter_of_row, scale,
               LA, ld_a, stride_a, order_a, LB, ld_b, stride_b, order_b, D, ldd, bias, activation,
               d_type, stream, check):
    ep = Epilogue(_addr(bias), int(activation), int(d_type))
    st = getattr(library(), fn_name)(
        int(M), int(N), int(K), _addr(X), int(ldx), _addr(W), int(ldw), int(order_w),
        int(adapters), int(rank), _addr(adapter_of_row), _addr(scale), _addr(LA), int(ld_a),
        int(stride_a), int(order_a), _addr(LB), int(ld_b), int(stride_b), int(order_b), _addr(D),
        int(ldd), ctypes.byref(ep), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, fn_name)
    return st


def gemm_lora_bf16_f32acc(M, N, K, X, ldx, W, ldw, order_w, adapters, rank, adapter_of_row, scale,
                          LA, ld_a, stride_a, order_a, LB, ld_b, stride_b, order_b, D, ldd,
                          bias=None, activation=GEMM_ACT_NONE, d_type=GEMM_D_F32, stream=None,
                          check=True) -> int:
    """A shared projection with each row's own low-rank adapter, BF16 (see include/gemm.h)."""
    return _call_lora("gemm_lora_bf16_f32acc", M, N, K, X, ldx, W, ldw, order_w, adapters, rank,
                      adapter_of_row, scale, LA, ld_a, stride_a, order_a, LB, ld_b, stride_b,
                      order_b, D, ldd, bias, activation, d_type, stream, check)


def gemm_lora_f16_f32acc(M, N, K, X, ldx, W, ldw, order_w, adapters, rank, adapter_of_row, scale,
                         LA, ld_a, stride_a, order_a, LB, ld_b, stride_b, order_b, D, ldd,
                         bias=None, activation=GEMM_ACT_NONE, d_type=GEMM_D_F32, stream=None,
                         check=True) -> int:
    """A shared projection with each row's own low-rank adapter, FP16 (see include/gemm.h)."""
    return _call_lora("gemm_lora_f16_f32acc", M, N, K, X, ldx, W, ldw, order_w, adapters, rank,
                      adapter_of_row, scale, LA, ld_a, stride_a, order_a, LB, ld_b, stride_b,
                      order_b, D, ldd, bias, activation, d_type, stream, check)


def gemm_probe_tc_bf16(cta_group, n_mma, stream=None, check=True):
    """Enqueue the tensor-pipe probe; returns (status, FLOPs of the launch)."""
    flops = ctypes.c_double(0.0)
    st = library().gemm_probe_tc_bf16(int(cta_group), int(n_mma), ctypes.byref(flops),
                                      _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_probe_tc_bf16")
    return st, flops.value


def gemm_probe_fma_f32(trips, stream=None, check=True):
    """Enqueue the FP32 FMA probe; returns (status, FLOPs of the launch)."""
    flops = ctypes.c_double(0.0)
    st = library().gemm_probe_fma_f32(int(trips), ctypes.byref(flops), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_probe_fma_f32")
    return st, flops.value


def gemm_probe_wait_timeout(timeout_ns, stream=None, check=True):
    """Enqueue the bounded-wait probe (a wait that runs out after timeout_ns)."""
    st = library().gemm_probe_wait_timeout(int(timeout_ns), _stream(stream))
    if check and st != GEMM_OK:
        raise GemmError(st, "gemm_probe_wait_timeout")
    return st


# ------------------------------------------------------------ torch helper
def storage_order(t):
    """(order, ld) of a 2-D tensor, from its strides; raises if neither dense-row nor dense-column."""
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor")
    r, q = t.shape
    s0, s1 = t.stride()
    if s1 == 1 and (s0 >= max(q, 1) or r <= 1):
        return ROW_MAJOR, max(s0, q, 1)
    if s0 == 1 and (s1 >= max(r, 1) or q <= 1):
        return COL_MAJOR, max(s1, r, 1)
    raise ValueError(f"tensor with strides {t.stride()} is neither row- nor column-major")


def gemm(A, B, C=None, alpha=1.0, beta=0.0, out=None, stream=None):
    """D = alpha * A @ B + beta * C for torch CUDA tensors.

    A (M x K) and B (K x N) are float32 (-> gemm_f32), bfloat16
    (-> gemm_bf16_f32acc) or float16 (-> gemm_f16_f32acc); C and the result
    are float32 and share one order
    (``out``'s if given, else C's, else row-major).  Any row- or
    column-major view works (e.g. ``B.t()`` of a contiguous N x K tensor).
    """
    import torch
    M, K = A.shape
    K2, N = B.shape
    if K2 != K:
        raise ValueError("inner dimensions differ")
    if A.dtype != B.dtype:
        raise TypeError("A and B must share a dtype")
    oa, lda = storage_order(A)
    ob, ldb = storage_order(B)
    if out is None:
        if C is not None and C.shape == (M, N):
            ocd_pref = storage_order(C)[0]
        else:
            ocd_pref = ROW_MAJOR
        out = torch.empty((M, N), dtype=torch.float32, device=A.device)
        if ocd_pref == COL_MAJOR:
            out = torch.empty((N, M), dtype=torch.float32, device=A.device).t()
    ocd, ldd = storage_order(out)
    ldc = ldd
    if beta != 0.0:
        if C is None:
            raise ValueError("beta != 0 needs C")
        oc, ldc = storage_order(C)
        if oc != ocd:
            raise ValueError("C and the output must share a storage order")
    fns = {torch.float32: gemm_f32, torch.bfloat16: gemm_bf16_f32acc,
           torch.float16: gemm_f16_f32acc}
    if A.dtype not in fns:
        raise TypeError("A and B must be float32, bfloat16 or float16")
    fn = fns[A.dtype]
    fn(M, N, K, alpha, A, lda, oa, B, ldb, ob, beta, C if beta != 0.0 else None, ldc, out, ldd,
       ocd, stream)
    return out


# ------------------------------------------------- torch helpers, grouped
# These run once per layer and token, beside kernels of a few microseconds, so
# they read each tensor attribute once and go straight to the C entry point.
# With `stream` the work goes to that stream and new outputs belong to its memory
# pool; as with torch's own operations, the caller orders the streams and calls
# record_stream for tensors that another stream than their own uses.
def stack_order(t):
    """(order, ld, stride) of a stack of matrices (3-D tensor), from its strides."""
    if t.dim() != 3:
        raise ValueError("expected a 3-D tensor (a stack of matrices)")
    n, r, q = t.shape
    s0, s1, s2 = t.stride()
    stride = s0 if n > 1 else 0
    if s2 == 1 and (s1 >= q or r <= 1):
        return ROW_MAJOR, max(s1, q, 1), stride
    if s1 == 1 and (s2 >= r or q <= 1):
        return COL_MAJOR, max(s2, r, 1), stride
    raise ValueError(f"tensor with strides {t.stride()} is neither row- nor column-major")


def _row_major(t, what):
    """Leading dimension of a row-major matrix, or of each matrix of a stack: the columns of a
    row are adjacent (one row has no pitch, one column no distance)."""
    *_, r, q = t.shape
    *_, s0, s1 = t.stride()
    if (s1 == 1 or q <= 1) and (s0 >= q or r <= 1):
        return max(s0, q, 1)
    raise ValueError(f"{what} must be row-major")


def _int_vector(t, n, what, device):
    """Address of a contiguous int32 vector of n."""
    if t.dtype is not _torch().int32:
        raise TypeError(f"{what} must be int32")
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous vector of {n}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    return t.data_ptr()


def _f32_dense(t, shape, what, device):
    """Address of a contiguous float32 tensor of this shape (None: None)."""
    if t is None:
        return None
    if t.dtype is not _torch().float32:
        raise TypeError(f"{what} must be float32")
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with shape {shape}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}")
    return t.data_ptr()


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_of(stream):
    if stream is not None:
        return _stream(stream)
    c = _torch()._C  # torch.cuda.current_stream().cuda_stream without its Python objects
    return c._cuda_getCurrentRawStream(c._cuda_getDevice())


def _empty_for(stream):
    """torch.empty for an output that `stream` (None: torch's current stream) writes: memory of
    that stream's pool, as work of another stream may still use what the current one's pool
    hands out."""
    torch = _torch()
    if stream is None:
        return torch.empty
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()

    def empty(*args, **kwargs):
        with torch.cuda.stream(stream):
            return torch.empty(*args, **kwargs)
    return empty


def _on_device(device):
    """Refuse operands that the kernels of the current device cannot read."""
    if device.type != "cuda":
        raise ValueError("the operands must be CUDA tensors")
    if device.index != _torch()._C._cuda_getDevice():
        raise ValueError(f"the operands are on {device}, which is not the current device")


def _types(A, B, out, out_dtype, default):
    """(entry point suffix, output dtype, d_type, device); A and B share a dtype, D is FP32 or that."""
    torch = _torch()
    dtype = A.dtype
    if B.dtype is not dtype:
        raise TypeError("the operands must share a dtype")
    device = A.device
    if B.device != device:
        raise ValueError("the operands must share a device")
    if dtype is torch.bfloat16:
        suffix, same = "bf16_f32acc", GEMM_D_BF16
    elif dtype is torch.float16:
        suffix, same = "f16_f32acc", GEMM_D_F16
    elif dtype is torch.float32:
        suffix, same = "f32", GEMM_D_F32
    else:
        raise TypeError("the operands must be float32, bfloat16 or float16")
    if out is not None:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError("out must have out_dtype")
        if out.device != device:
            raise ValueError("out must be on the operands' device")
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = default or dtype
    if out_dtype is dtype:
        return suffix, out_dtype, same, device
    if out_dtype is torch.float32:
        return suffix, out_dtype, GEMM_D_F32, device
    raise TypeError("the output must be float32 or the operands' dtype")


def group_rows(ids, groups, stream=None):
    """(offsets, order, position) of rows grouped by the int32 numbers `ids` (gemm_group_rows)."""
    torch = _torch()
    device, n = ids.device, ids.numel()
    at = _int_vector(ids, n, "ids", device)
    _on_device(device)
    # (views of one allocation would cost the host more than three allocations)
    empty = _empty_for(stream)
    offsets = empty(groups + 1, dtype=torch.int32, device=device)
    order = empty(n, dtype=torch.int32, device=device)
    position = empty(n, dtype=torch.int32, device=device)
    st = library().gemm_group_rows(n, groups, at, offsets.data_ptr(), order.data_ptr(),
                                   position.data_ptr(), _stream_of(stream))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_group_rows")
    return offsets, order, position


def gemm_grouped(A, B, offsets, row_index=None, bias=None, activation=GEMM_ACT_NONE,
                 out_dtype=None, out=None, alpha=1.0, stream=None):
    """D[r] = act(alpha * A[idx(r)] @ B[g] + bias[g]) for the rows r of each group g.

    A is (rows_a x K) row-major, B a stack (groups x K x N) of row- or
    column-major matrices (e.g. ``W.transpose(1, 2)`` of groups x N x K
    weights), offsets int32 (groups + 1) on the device; row_index int32 gathers
    the rows of A (one per row of D).  D is float32 or the operands' dtype
    (the default).  Rows of D outside every group are left as they are.
    """
    suffix, out_dtype, d_type, device = _types(A, B, out, out_dtype, None)
    order_b, ldb, stride_b = stack_order(B)
    groups, K, N = B.shape
    if A.dim() != 2 or A.shape[1] != K:
        raise ValueError("inner dimensions differ")
    rows_a = rows = A.shape[0]
    lda = _row_major(A, "A")
    index = None
    if row_index is not None:
        rows = row_index.shape[0]
        index = _int_vector(row_index, rows, "row_index", device)
    at = _int_vector(offsets, groups + 1, "offsets", device)
    ep = Epilogue(_f32_dense(bias, (groups, N), "bias", device), activation, d_type)
    if out is not None and tuple(out.shape) != (rows, N):
        raise ValueError(f"out must be {rows} x {N}")
    _on_device(device)
    if out is None:
        out = _empty_for(stream)((rows, N), dtype=out_dtype, device=device)
        ldd = N
    else:
        ldd = _row_major(out, "out")
    fn = "gemm_grouped_" + suffix
    st = getattr(library(), fn)(groups, rows, N, K, alpha, A.data_ptr(), lda, rows_a, index, at,
                                B.data_ptr(), ldb, stride_b, order_b, out.data_ptr(), ldd, ep,
                                _stream_of(stream))
    if st != GEMM_OK:
        raise GemmError(st, fn)
    return out


def gemm_grouped_wgrad(A, B, offsets, row_index=None, C=None, alpha=1.0, beta=0.0, out_dtype=None,
                       out=None, stream=None):
    """D[g] = alpha * A[idx(rows of g)].T @ B[rows of g] + beta * C[g], a stack (groups x M x N).

    A is (rows_a x M), B (rows x N), both row-major; offsets and row_index as
    for ``gemm_grouped``.  D is float32 (the default) or the operands' dtype, C
    float32.  Groups without rows give beta * C[g].
    """
    torch = _torch()
    suffix, out_dtype, d_type, device = _types(A, B, out, out_dtype, torch.float32)
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be matrices")
    (rows_a, M), (rows, N), groups = A.shape, B.shape, offsets.shape[0] - 1
    lda, ldb = _row_major(A, "A"), _row_major(B, "B")
    at = _int_vector(offsets, groups + 1, "offsets", device)
    index = None
    if row_index is not None:
        index = _int_vector(row_index, rows, "row_index", device)
    elif rows_a != rows:
        raise ValueError("A and B must have as many rows")

    def stack(t, what):
        if tuple(t.shape) != (groups, M, N):
            raise ValueError(f"{what} must be {groups} x {M} x {N}")
        return _row_major(t, what), t.stride(0) if groups > 1 else 0

    if out is not None:
        ldd, stride_d = stack(out, "out")
    c, ldc, stride_c = None, 0, 0
    if beta != 0.0:
        if C is None:
            raise ValueError("beta != 0 needs C")
        if C.dtype is not torch.float32:
            raise TypeError("C must be float32")
        if C.device != device:
            raise ValueError("C must be on the operands' device")
        ldc, stride_c = stack(C, "C")
        c = C.data_ptr()
    _on_device(device)
    if out is None:
        out = _empty_for(stream)((groups, M, N), dtype=out_dtype, device=device)
        ldd, stride_d = max(N, 1), M * N
    fn = "gemm_grouped_wgrad_" + suffix
    st = getattr(library(), fn)(groups, rows, M, N, alpha, A.data_ptr(), lda, rows_a, index, at,
                                B.data_ptr(), ldb, beta, c, ldc, stride_c, out.data_ptr(), ldd,
                                stride_d, d_type, _stream_of(stream))
    if st != GEMM_OK:
        raise GemmError(st, fn)
    return out


def gemm_lora(X, W, LA, LB, adapter_of_row, scale=None, bias=None, activation=GEMM_ACT_NONE,
              out_dtype=None, out=None, stream=None):
    """D[i] = act(X[i] @ W + scale[a] * (X[i] @ LA[a]) @ LB[a] + bias), a = adapter_of_row[i].

    X is (M x K) row-major, W (K x N), LA a stack (adapters x K x rank), LB a
    stack (adapters x rank x N), each row- or column-major, all bfloat16 or
    all float16; adapter_of_row int32 (a number outside [0, adapters): no
    adapter), scale float32 per adapter.  D is float32 or the operands' dtype
    (the default).
    """
    suffix, out_dtype, d_type, device = _types(X, W, out, out_dtype, None)
    if suffix == "f32":
        raise TypeError("gemm_lora takes bfloat16 or float16")
    if LA.dtype is not X.dtype or LB.dtype is not X.dtype:
        raise TypeError("the operands must share a dtype")
    if LA.device != device or LB.device != device:
        raise ValueError("the operands must share a device")
    order_a, ld_a, stride_a = stack_order(LA)
    order_b, ld_b, stride_b = stack_order(LB)
    (M, K), (kw, N), (adapters, ka, rank) = X.shape, W.shape, LA.shape
    if kw != K or ka != K:
        raise ValueError("inner dimensions differ")
    if tuple(LB.shape) != (adapters, rank, N):
        raise ValueError(f"LB must be {adapters} x {rank} x {N}")
    ldx = _row_major(X, "X")
    order_w, ldw = storage_order(W)
    ids = _int_vector(adapter_of_row, M, "adapter_of_row", device)
    scales = _f32_dense(scale, (adapters,), "scale", device)
    ep = Epilogue(_f32_dense(bias, (N,), "bias", device), activation, d_type)
    if out is not None and tuple(out.shape) != (M, N):
        raise ValueError(f"out must be {M} x {N}")
    _on_device(device)
    if out is None:
        out = _empty_for(stream)((M, N), dtype=out_dtype, device=device)
        ldd = N
    else:
        ldd = _row_major(out, "out")
    fn = "gemm_lora_" + suffix
    st = getattr(library(), fn)(M, N, K, X.data_ptr(), ldx, W.data_ptr(), ldw, order_w, adapters,
                                rank, ids, scales, LA.data_ptr(), ld_a, stride_a, order_a,
                                LB.data_ptr(), ld_b, stride_b, order_b, out.data_ptr(), ldd, ep,
                                _stream_of(stream))
    if st != GEMM_OK:
        raise GemmError(st, fn)
    return out
