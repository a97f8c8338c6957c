"""Shared plumbing of the grouped operators' tests: inputs, the definitions in
64 bits (numpy loops over groups, no code of the library) and tolerances.

Tolerance of a sum of K products of the inputs, S = sum |a b|: the tensor
cores add 16 products and the accumulator per step, 17 addends aligned to the
largest and cut to FP32's 24 bits, so each of ceil(K / 16) steps is off by at
most 18 * 2^-23 of the largest partial sum, itself at most S; the CUDA-core
kernels' K sequential roundings of 2^-24 stay below that.  A 16-bit D adds half
an ulp (2^-8 relative for BF16, 2^-11 and the subnormal step 2^-24 for FP16),
an FP32 D 2^-23 for the epilogue's own roundings.  GELU's slope is at most 1.13
and its tanhf within 1e-6 of the value.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import dense_gemm_08_gb300 as lib

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SUFFIX = {"f32": "f32", "bf16": "bf16_f32acc", "f16": "f16_f32acc"}
D_TYPE = {"f32": lib.GEMM_D_F32, "bf16": lib.GEMM_D_BF16, "f16": lib.GEMM_D_F16}
SENTINEL = 1234.0


def rel_sum(K):
    return 18 * math.ceil(max(K, 1) / 16) * 2.0 ** -23


def rounding(out, ref):
    a = np.abs(ref)
    if out == "bf16":
        return a * 2.0 ** -8
    if out == "f16":
        return a * 2.0 ** -11 + 2.0 ** -24
    return a * 2.0 ** -22


def draw(rng, shape, dtype, dist="normal", sigma=1.0):
    if dist == "int":
        x = rng.integers(-3, 4, shape).astype(np.float32)
    else:
        x = (rng.standard_normal(shape) * sigma).astype(np.float32)
    return torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def padded(t, pad_to, extra=0, fill=float("nan")):
    """The same values with the innermost extent stored padded (fill in the padding)."""
    n = t.shape[-1]
    ld = -(-n // pad_to) * pad_to + extra
    buf = torch.full((*t.shape[:-1], ld), fill, dtype=t.dtype)
    buf[..., :n] = t
    return buf.cuda()[..., :n]


def offsets_of(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def activate(z, act):
    if act == lib.GEMM_ACT_RELU:
        return np.maximum(z, 0.0)
    if act == lib.GEMM_ACT_GELU:
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def gathered(A, row_index):
    a = f64(A)
    if row_index is None:
        return a
    idx = row_index.cpu().numpy()
    out = np.zeros((len(idx), a.shape[1]))
    ok = (idx >= 0) & (idx < a.shape[0])
    out[ok] = a[idx[ok]]
    return out


def grouped_ref(A, B, offsets, row_index, bias, act, alpha):
    """(D, tolerance before D's rounding, rows inside a group) of the grouped product."""
    a, b = gathered(A, row_index), f64(B)
    rows, N = a.shape[0], b.shape[2]
    D, tol = np.zeros((rows, N)), np.zeros((rows, N))
    inside = np.zeros(rows, dtype=bool)
    for g in range(b.shape[0]):
        lo = min(max(int(offsets[g]), 0), rows)
        hi = min(max(int(offsets[g + 1]), lo), rows)
        z = alpha * (a[lo:hi] @ b[g])
        S = abs(alpha) * (np.abs(a[lo:hi]) @ np.abs(b[g]))
        t = rel_sum(a.shape[1]) * S + 2.0 ** -22 * np.abs(z)
        if bias is not None:
            z = z + f64(bias)[g]
            t = t + 2.0 ** -22 * (np.abs(z) + np.abs(f64(bias)[g]))
        y = activate(z, act)
        if act == lib.GEMM_ACT_GELU:
            t = 1.13 * t + 1e-6 * np.abs(z) + 1e-6
        D[lo:hi], tol[lo:hi] = y, t
        inside[lo:hi] = True
    return D, tol, inside


def wgrad_ref(A, B, offsets, row_index, C, alpha, beta):
    a, b = gathered(A, row_index), f64(B)
    groups = len(offsets) - 1
    rows, M, N = b.shape[0], a.shape[1], b.shape[1]
    D, tol = np.zeros((groups, M, N)), np.zeros((groups, M, N))
    for g in range(groups):
        lo = min(max(int(offsets[g]), 0), rows)
        hi = min(max(int(offsets[g + 1]), lo), rows)
        D[g] = alpha * (a[lo:hi].T @ b[lo:hi])
        tol[g] = rel_sum(hi - lo) * abs(alpha) * (np.abs(a[lo:hi]).T @ np.abs(b[lo:hi]))
        tol[g] += 2.0 ** -22 * np.abs(D[g])
        if beta:
            c = beta * f64(C)[g]
            D[g] += c
            tol[g] += 2.0 ** -22 * (np.abs(c) + np.abs(D[g]))
    return D, tol


def lora_ref(X, W, LA, LB, ids, scale, bias, act, dtype, out):
    """The second product's first operand is rounded to the inputs' type (16-bit D) or to two
    such values (FP32 D): 2^-9 / 2^-12 relative, or 2^-17 / 2^-23 (twice that is allowed)."""
    x, w, la, lb = f64(X), f64(W), f64(LA), f64(LB)
    ids = ids.cpu().numpy()
    unit = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    if out == "f32":
        unit = {"bf16": 2.0 ** -16, "f16": 2.0 ** -21}[dtype]
    z = x @ w
    tol = rel_sum(x.shape[1]) * (np.abs(x) @ np.abs(w))
    n, r = la.shape[0], la.shape[2]
    for i, a in enumerate(ids):
        if 0 <= a < n:
            s = 1.0 if scale is None else float(scale[a])
            u = s * (x[i] @ la[a])
            su = abs(s) * (np.abs(x[i]) @ np.abs(la[a]))
            z[i] += u @ lb[a]
            big = np.abs(lb[a])
            tol[i] += (rel_sum(x.shape[1]) * su + (unit + rel_sum(r)) * np.abs(u) + 2.0 ** -24) @ big
    tol += 2.0 ** -22 * np.abs(z)
    if bias is not None:
        z = z + f64(bias)
        tol = tol + 2.0 ** -22 * (np.abs(z) + np.abs(f64(bias)))
    y = activate(z, act)
    if act == lib.GEMM_ACT_GELU:
        tol = 1.13 * tol + 1e-6 * np.abs(z) + 1e-6
    return y, tol


def assert_close(got, ref, tol, out, what=""):
    got = got.detach().cpu().to(torch.float64).numpy()
    bound = tol * (1 + 2.0 ** -8) + rounding(out, ref)
    bad = ~(np.abs(got - ref) <= bound)
    if bad.any():
        at = np.argwhere(bad)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound, first "
                             f"{at[:4].tolist()}, last {at[-1].tolist()}, got "
                             f"{got[tuple(at[0])]:.6g} for {ref[tuple(at[0])]:.6g}")


def done():
    torch.cuda.synchronize()
    assert lib.gemm_last_device_status() == lib.GEMM_OK
