"""The router's choice in 64 bits, whole batches at once, and where 64 bits decide it.

A score in 64 bits is off by a few units of 2^-53 of itself: exp and a division by one unit each, a
sum of at most 1024 terms by 10 halvings, and c = s + b by half a unit of s + |b|.  Two values further
apart than 2^-47 of the larger s + |b| (64 units of 2^-53) are in the same order however
they are computed, sums of two of them as well; nearer ones are in doubt, unless their logits and
biases are the same: then they are equal in any arithmetic, and the lower index comes first.  An expert whose logit
or bias is -infinity is out of the choice, whatever its other value is."""
import numpy as np

from mixture_harness import scores

DOUBT = 2.0 ** -47


def _falling(v):
    """Order of the last axis by falling value, a NaN first, equal ones by index."""
    nan = np.isnan(v)
    return np.lexsort((-np.where(nan, 0.0, v), ~nan), axis=-1)  # (stable; a NaN before +infinity)


def _in_doubt(a, b, size, same):
    """a comes before b, but may not: they are finite, too near and not of the same inputs."""
    with np.errstate(invalid="ignore"):
        return np.isfinite(a) & np.isfinite(b) & (a - b <= DOUBT * size) & ~same


def choice(x, k, score, bias=None, groups=1, kept=1, top=1):
    """(chosen [T, k] (-1: none), sure [T]: no decision of the token is in doubt)."""
    T, E = x.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    masked = (x == -np.inf) | (b == -np.inf)
    with np.errstate(invalid="ignore"):
        s = scores(x, score)
        c = x if bias is None else s + b
        mag = np.where(masked | ~np.isfinite(s + np.abs(b)), 0.0, s + np.abs(b))
    c = np.where(masked, -np.inf, c)
    by = np.where(masked, -np.inf, s) if bias is None and top == 2 else c
    exact = bias is None  # then c is the logit itself
    sure = np.ones(T, dtype=bool)
    out = masked.copy()
    if groups > 1 and kept < groups:
        size = E // groups
        v = by.reshape(T, groups, size)
        first = np.argsort(_falling(v), axis=-1, kind="stable") < min(top, size)  # (ranks)
        with np.errstate(invalid="ignore"):
            g = np.where(first & (v != -np.inf), v, 0.0).sum(-1)
        g = np.where((v == -np.inf).all(-1), -np.inf, g)
        order = _falling(g)
        stays = np.argsort(order, axis=-1, kind="stable") < kept
        stays &= g != -np.inf
        out |= ~np.repeat(stays, size, axis=1)
        if not (exact and top == 1):
            last = np.take_along_axis(order, np.full((T, 1), kept - 1), 1)
            then = np.take_along_axis(order, np.full((T, 1), kept), 1)
            at = np.arange(T)[:, None]
            # of the same inputs: the pairs (logit, bias) of their largest ones agree
            pair = np.stack([np.where(first, x.reshape(T, groups, size), -np.inf),
                             np.where(first, np.broadcast_to(b, x.shape).reshape(T, groups, size), 0.0)], -1)
            rank = np.argsort(-pair[..., 0], axis=-1, kind="stable")[..., None]
            pair = np.take_along_axis(pair, np.broadcast_to(rank, pair.shape), 2)[:, :, :2]
            same = (pair[at, last] == pair[at, then]).reshape(T, -1).all(1)
            most = np.where(first, mag.reshape(T, groups, size), 0.0).sum(-1).max(-1)
            sure &= ~_in_doubt(g[at, last][:, 0], g[at, then][:, 0], most, same)
    c = np.where(out, -np.inf, c)
    order = _falling(c)
    chosen = order[:, :k].copy()
    chosen[np.take_along_axis(c, chosen, 1) == -np.inf] = -1
    if not exact:
        at = order[:, :k + 1]
        v, size = np.take_along_axis(c, at, 1), np.take_along_axis(mag, at, 1)
        xs, bs = np.take_along_axis(x, at, 1), b[at]
        same = (xs[:, :-1] == xs[:, 1:]) & (bs[:, :-1] == bs[:, 1:])
        sure &= ~_in_doubt(v[:, :-1], v[:, 1:], np.maximum(size[:, :-1], size[:, 1:]), same).any(1)
    return chosen, sure
