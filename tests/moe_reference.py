"""Plain expert routing, token exchange and activations on the CPU in 64 bits, with what the kernels'
arithmetic may be off by.  Test infrastructure only."""
import math

import numpy as np

EPS = 2.0 ** -24  # half a step of fp32, relative


def route(logits, k, valid=None, normalize=True):
    """logits fp64 [T, E].  A dict of numpy arrays as moe_route writes them (token: -1 behind the last row), with p (softmax
    of the tokens that have an expert) and total (sum of a token's chosen p)."""
    T, E = logits.shape
    l = np.where(np.isnan(logits), -np.inf, logits)
    if valid is not None:
        l[~np.asarray(valid, bool)] = -np.inf
    expert = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int64)
    has = np.take_along_axis(l, expert, 1) > -np.inf
    expert = np.where(has, expert, -1)
    p, w, total = np.zeros((T, E)), np.zeros((T, k)), np.ones(T)
    for t in np.nonzero(has[:, 0])[0]:
        with np.errstate(invalid="ignore"):
            e = np.exp(logits[t] - l[t].max())
            p[t] = e / e.sum()
        w[t, has[t]] = p[t, expert[t, has[t]]]
        total[t] = w[t].sum()
        if normalize:
            w[t] /= total[t]
    counts = np.bincount(expert[has], minlength=E).astype(np.int64)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    position, token, at = np.full((T, k), -1), np.full(T * k, -1), offsets[:-1].copy()
    for t in range(T):
        for j in range(k):
            if has[t, j]:
                position[t, j] = at[expert[t, j]]
                token[position[t, j]] = t
                at[expert[t, j]] += 1
    n, c = int(has[:, 0].sum()), int(counts.sum())
    slope = E * counts / (c * n) if n else np.zeros(E)
    return dict(expert=expert, weight=w, counts=counts, offsets=offsets, position=position, token=token, p=p, total=total,
                slope=slope, loss=float((slope * p.sum(0)).sum()), has=has)


def route_error(logits, r):
    """Relative error of p and weights, one figure a token: the difference l - max is rounded (2^-24 of it) before the
    exponential (2 ulp), numerator and denominator each; a sum of E positive terms over at most 32 sequential adds and
    10 tree levels; a division, a product."""
    with np.errstate(invalid="ignore"):
        d = np.where(np.isfinite(logits), np.nanmax(np.where(np.isfinite(logits), logits, -1e30), 1, keepdims=True) - logits, 0.0)
    return (2 * np.minimum(d.max(1), 110.0) + 80) * EPS


def route_grad(r, dweight, dloss, normalize=True):
    """(dlogits, the magnitudes that its errors scale with)."""
    T, E = r["p"].shape
    dw = np.where(r["has"], dweight, 0.0) if dweight is not None else np.zeros(r["has"].shape)
    size = np.abs(dw)
    if normalize:
        size = np.where(r["has"], (size + (size * r["weight"]).sum(1, keepdims=True)) / r["total"][:, None], 0.0)
        dw = np.where(r["has"], (dw - (dw * r["weight"]).sum(1, keepdims=True)) / r["total"][:, None], 0.0)
    dp = np.tile(dloss * r["slope"], (T, 1))
    A = np.abs(dp)
    for j in range(dw.shape[1]):
        t = np.nonzero(r["has"][:, j])[0]
        dp[t, r["expert"][t, j]] += dw[t, j]
        A[t, r["expert"][t, j]] += size[t, j]
    p = r["p"]
    return p * (dp - (p * dp).sum(1, keepdims=True)), p * (A + (p * A).sum(1, keepdims=True))


GELU, SILU, GEGLU, SWIGLU = range(4)


def act(a, kind):
    """act(a), its derivative, and what each may be off by in the kernels' fp32 (absolute)."""
    a = np.asarray(a, np.float64)
    if kind in (GELU, GEGLU):
        cdf = 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(-a / math.sqrt(2))
        phi = np.exp(-a * a / 2) / math.sqrt(2 * math.pi)
        y, d = a * cdf, cdf + a * phi
        # Phi within 3e-7 (formula 26.2.17 and the hardware's 2^x and 1/x); the density's exponent is rounded three
        # times (3 a^2 / 2 units of 2^-24), 2^x is good to 2^-22; a few roundings of the results
        return y, d, 3e-7 * np.abs(a) + 4 * EPS * np.abs(y), 3e-7 + 8 * EPS + np.abs(a) * phi * (6 + 3 * a * a) * EPS
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-a))
    y, d = a * s, s * (1 + a * (1 - s))
    # exp(-a) = 2^(-a log2 e): two roundings of the exponent (2 |a| units of 2^-24), 2^x good to 2^-22, 1/x to 2^-23, an add,
    # a product: r, relative, for s and y.  1 - s is off by r s + 2^-24; times a, plus 1, times s: 2 r s (1 + |a|) + 4 units.
    # Values below 2^-126 are flushed to zero.
    r = (2 * np.abs(a) + 9) * EPS
    return y, d, r * np.abs(y) + 2.0 ** -118, 2 * r * s * (1 + np.abs(a)) + 4 * EPS + 2.0 ** -118
