"""Shared plumbing of the router's, the combination's and the fused products'
tests: the definitions in 64 bits (numpy, no code of the library) and
tolerances, each derived where it stands."""
from __future__ import annotations

import math

import numpy as np
import torch

import dense_gemm_08_gb300 as lib
from grouped_harness import D_TYPE, SUFFIX, TORCH, f64, padded, rel_sum  # noqa: F401

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a rounding, relative
LEAST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}  # below: absolute steps


def stored(x, dtype, extra=0, fill=float("nan")):
    """A CUDA tensor of the values, its rows padded by `extra` values of `fill`."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype])
    if not extra:
        return t.cuda()
    buf = torch.full((*t.shape[:-1], t.shape[-1] + extra), fill, dtype=t.dtype)
    buf[..., :t.shape[-1]] = t
    return buf.cuda()[..., :t.shape[-1]]


def rounding(dtype, ref):
    """Half a step of the type at the value (fp16: also of its subnormals)."""
    return np.abs(ref) * HALF_STEP[dtype] + LEAST[dtype]


# ------------------------------------------------------------------- router
def scores(x, score):
    with np.errstate(all="ignore"):
        if score == lib.GEMM_SCORE_SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        m = np.fmax.reduce(x, axis=-1, keepdims=True)
        e = np.where(x == -np.inf, 0.0, np.exp(x - m))
        return e / e.sum(-1, keepdims=True)


def _rank(values):
    """Indices by falling value, NaN first, equal ones by index."""
    nan = np.isnan(values)
    return sorted(range(len(values)),
                  key=lambda i: (0, 0.0, i) if nan[i] else (1, -values[i], i))


def route_ref(x, k, score, bias, groups, kept, top, renorm, scale):
    """(chosen, weights) from logits in 64 bits."""
    T, E = x.shape
    s = scores(x, score)
    chosen, weights = np.full((T, k), -1), np.zeros((T, k))
    for t in range(T):
        masked = x[t] == -np.inf
        c = x[t].copy() if bias is None else s[t] + bias
        c[masked] = -np.inf
        by = s[t].copy() if bias is None and top == 2 else c.copy()
        by[masked] = -np.inf
        allowed = np.ones(E, dtype=bool)
        if groups > 1 and kept < groups:
            size = E // groups
            score_of = []
            for g in range(groups):
                v = by[g * size:(g + 1) * size]
                best = [v[i] for i in _rank(v)[:top] if v[i] != -np.inf]
                score_of.append(sum(best) if best else -np.inf)
            allowed[:] = False
            for g in [g for g in _rank(np.array(score_of)) if score_of[g] != -np.inf][:kept]:
                allowed[g * size:(g + 1) * size] = True
        ids = [e for e in _rank(c) if allowed[e] and c[e] != -np.inf][:k]
        chosen[t, :len(ids)] = ids
        w = s[t, ids]
        if renorm and ids:
            with np.errstate(all="ignore"):
                total = w.sum()
                if total < 1e-30 and score == lib.GEMM_SCORE_SIGMOID:  # ratios survive
                    l = np.minimum(x[t, ids], 0) - np.log1p(np.exp(-np.abs(x[t, ids])))
                    w = np.exp(l - l.max())
                    total = w.sum()
                w = w / total
        weights[t, :len(ids)] = w * scale
    return chosen, weights


def route_grad_ref(x, chosen, dw, score, renorm, scale):
    """dlogits by the chain rule, through the scores' Jacobian."""
    T, E = x.shape
    s = scores(x, score)
    out = np.zeros((T, E))
    for t in range(T):
        has = [(j, e) for j, e in enumerate(chosen[t]) if 0 <= e < E]
        ds = np.zeros(E)
        total = sum(s[t, e] for _, e in has)
        for j, e in has:
            if renorm:
                ds[e] += scale * dw[t, j] / total
                for _, o in has:
                    ds[o] -= scale * dw[t, j] * s[t, e] / total ** 2
            else:
                ds[e] += scale * dw[t, j]
        if score == lib.GEMM_SCORE_SIGMOID:
            out[t] = ds * s[t] * (1 - s[t])
        else:
            out[t] = s[t] * (ds - (ds * s[t]).sum())
    return out


# ------------------------------------------------------------ fused products
def activation(z, act):
    with np.errstate(all="ignore"):
        if act == lib.GEMM_ACT_RELU:
            return np.where(z <= 0, 0.0, z)
        if act == lib.GEMM_ACT_GELU:
            return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
        if act == lib.GEMM_ACT_SILU:
            return z / (1 + np.exp(-z))
    return z


def slope(z, act):
    with np.errstate(all="ignore"):
        if act == lib.GEMM_ACT_RELU:
            return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
        if act == lib.GEMM_ACT_GELU:
            c = math.sqrt(2 / math.pi)
            t = np.tanh(c * (z + 0.044715 * z ** 3))
            return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
        if act == lib.GEMM_ACT_SILU:
            s = 1 / (1 + np.exp(-z))
            return s * (1 + z * (1 - s))
    return np.ones_like(z)


def act_error(dtype, z):
    """Of the activation in FP32, on top of Z's own.  x times a logistic function of an argument a:
    exp(-|a|) is off by 2 + 1.2 |a| units of 2^-23 (16-bit types: the hardware's; expf: 2), a's own
    three roundings move it by |a| 2^-22, the division and products add 4 units; relative to
    the value where x > 0 (a exp(-a) < 0.4), and below 2^-20 where x < 0 as |x| exp(-|a|) (6 +
    2.2 |a|) 2^-23 < 8 * 2^-23."""
    return 2.0 ** -20 * np.abs(z) + 2.0 ** -20


SLOPE_ERROR = 2.0 ** -18  # the same, with x times its slope at most 1.2 in place of |x| exp(-|a|)
STEEP = 1.13  # the largest slope of GELU; SiLU's is 1.1


def product(A, B, alpha):
    """(alpha A B, bound of its error) in 64 bits."""
    a, b = f64(A), f64(B)
    z = alpha * (a @ b)
    return z, rel_sum(a.shape[1]) * abs(alpha) * (np.abs(a) @ np.abs(b)) + 2.0 ** -22 * np.abs(z)


def fused_ref(A, B, bias, act, residual, alpha, dtype):
    """(D, its tolerance, Z, its tolerance)."""
    z, tol = product(A, B, alpha)
    if bias is not None:
        b = f64(bias)
        z = z + b
        tol = tol + 2.0 ** -23 * (np.abs(z) + np.abs(b))
    d, dtol = activation(z, act), tol
    if act in (lib.GEMM_ACT_GELU, lib.GEMM_ACT_SILU):
        dtol = STEEP * tol + act_error(dtype, z)
    if residual is not None:
        r = f64(residual)
        d = d + r
        dtol = dtol + 2.0 ** -23 * (np.abs(d) + np.abs(r))
    return (d, dtol * (1 + HALF_STEP[dtype]) + rounding(dtype, d),
            z, tol * (1 + HALF_STEP[dtype]) + rounding(dtype, z))


def fused_grad_ref(A, B, pre, act, alpha, dtype):
    """(D, its tolerance, dbias, its tolerance)."""
    g, tol = product(A, B, alpha)
    if act != lib.GEMM_ACT_NONE:
        z = f64(pre)
        f = slope(z, act)
        tol = tol * np.abs(f) + np.abs(g) * (2.0 ** -23 * np.abs(f))
        if act != lib.GEMM_ACT_RELU:
            tol = tol + np.abs(g) * SLOPE_ERROR
        g = g * f
    # a column's sum: each D's error, and one rounding per addition of partial sums that are at most
    # sum |D| (blocks of rows, then blocks: at most 64 + log2-like steps each, 200 in all)
    dbias = g.sum(0)
    btol = tol.sum(0) + 200 * 2.0 ** -24 * np.abs(g).sum(0) + 1e-30
    return g, tol * (1 + HALF_STEP[dtype]) + rounding(dtype, g), dbias, btol


def check(got, ref, tol, what=""):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, what
    same = np.isnan(got) & np.isnan(ref) | (got == ref)
    bad = ~same & ~(np.abs(got - ref) <= tol)
    if bad.any():
        at = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first {at}: got {got[at]!r}, "
                             f"want {ref[at]!r}, tolerance {np.broadcast_to(tol, ref.shape)[at]!r}")
