"""Sampling from its definition in 64 bits on the host.

A weight of the kernel is off by a relative error of at most 2 |t| U (t = (logit - max) / temperature log2 e: the
difference, the product) + 4 U (the exponential's unit, its argument's last rounding), U = 2^-24; sums over a
wavefront's pieces in 32 bits add 14 U (8 elements, 6 sums over lanes).  Shares of the sum are then off by no more than twice the mean of that over the
kept weights, and a border (a share that top-p or the random number is compared with, or a weight next to min_p)
may fall on the other side only if it lies closer than that."""
import numpy as np

U = 2.0 ** -24


def token(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row z (float64), and the error of shares of the kept weights."""
    z = np.where(np.isnan(z), -np.inf, z)
    most = z.max() if z.size else -np.inf
    if most == -np.inf:
        return -1, 0.0
    if not temperature > 0:
        return int(np.argmax(z)), 0.0
    with np.errstate(invalid="ignore", over="ignore"):
        t = np.where(z == most, 0.0, -np.inf if most == np.inf else (z - most) / temperature)
    w = np.exp(t)
    keep = np.isfinite(t) | (t == 0)
    if 0 < top_k < z.size or top_p < 1:
        order = np.argsort(-z, kind="stable")
        order = order[keep[order]]
        if 0 < top_k < z.size:
            order = order[:top_k]
        if top_p < 1:
            run = np.cumsum(w[order])
            before = np.concatenate([[0.0], run[:-1]])
            order = order[(before < top_p * run[-1]) | (np.arange(order.size) == 0)]
        keep = np.zeros(z.size, bool)
        keep[order] = True
    w = np.where(keep & (w >= min(min_p, 1.0)), w, 0.0)
    run = np.cumsum(w)
    u = 0.0 if not u > 0 else min(u, 1.0)
    over = run > u * run[-1]
    i = int(np.argmax(over)) if over.any() else int(np.nonzero(w)[0][-1])
    depth = np.where(w > 0, np.abs(np.where(np.isfinite(t), t, 0.0)), 0.0) * 1.4427
    return i, float(2 * (w * (2 * depth + 18) * U).sum() / run[-1])


def accepted(z, u, got, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Whether `got` is the token, or one that the error of the weights allows."""
    args = (temperature, top_k)
    want, e = token(z, u, *args, top_p, min_p)
    if got == want:
        return True
    for p in (top_p, top_p - e, top_p + e) if top_p < 1 else (top_p,):
        for m in (min_p, min_p * (1 - 64 * U), min_p * (1 + 64 * U)) if min_p > 0 else (min_p,):
            for v in (u - e, u, u + e):
                if got == token(z, v, *args, p, m)[0]:
                    return True
    return False
