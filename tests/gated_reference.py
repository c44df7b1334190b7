"""The gated linear recurrence from its formulas in 64 bits on the host, row by row, with the error that 32-bit
arithmetic may make.

    f = sigmoid(decay), g = sigmoid(input), z = rate f, a = exp(z), w = sqrt(1 - a^2), h[t] = a h[t-1] + w g x

Roundings counted (U = 2^-24 each; exp2, reciprocal and roots of the hardware are good to one unit in the last
place, 2 U), first order, relative unless said otherwise:
    f, g        e^-u by exp2(-u log2 e): 2 U |u| (constant and product) + 2 U; 1 + e: U; the reciprocal: 2 U
    1 - f       e^-u f: f's, e^-u's and U
    a           z's error and 2 U (constant and product), times |z|; exp2: 2 U
    1 - a^2     at most 1.2 times the errors of a and z (its slope by z is at most 1, -2 a z and the series carry a's
                and z's along; fma(-a, a, 1) carries 2 a^2 / (1 - a^2) <= 1.17 of a's), and 5 U
    w           half of that, and 2 U
    h           the recurrence carries the error of a row on as it carries the row: e[t] = a e[t-1] + ...; maps of
                several rows composed round once more per row (the product of factors, and a few sums per eight rows)
Where a sigmoid or the factor a is below 2^-125, the hardware's reciprocal or exponential may flush it to zero (results
below 2^-126): all of its value is counted as an error.  (A factor of 5.5e-39 times a rate of 200 is 1.1e-36 of the
state in ddecay, above the type's smallest normal number.)"""
import numpy as np

import sequence_reference as ref

U = ref.U


def sigmoid(v):
    """Without an overflow of the exponential."""
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def product(p, pe, q, qe, roundings=1):
    return np.abs(p) * qe + np.abs(q) * pe + roundings * U * np.abs(p * q)


def gated(x, decay, inp, rate, seqs, initial=None, dy=None, dfinal=None):
    """{name: (value, error before the final rounding)}; x, decay, inp, dy (rows, D), rate (D,), states (S, D)."""
    rows, d = x.shape
    f, g = sigmoid(decay), sigmoid(inp)
    rf = np.where(f < 2.0 ** -125, 1.5, (2 * np.abs(decay) + 5) * U)
    rg = np.where(g < 2.0 ** -125, 1.5, (2 * np.abs(inp) + 5) * U)
    z = rate * f
    rz = rf + U
    a = np.exp(z)
    ra = np.where(a < 2.0 ** -125, 1.5, np.abs(z) * (rz + 2 * U) + 2 * U)
    w2 = -np.expm1(2 * z)
    w = np.sqrt(w2)
    rw = 0.6 * (np.abs(z) * (rz + 2 * U) * (a >= 2.0 ** -125) + 2 * U + rz) + 4.5 * U  # 1 - a^2 is 1 where a is flushed
    b = w * g * x
    b_e = (rw + rg + 2 * U) * np.abs(b)
    h, m, e, before, before_m, before_e = (np.zeros((rows, d)) for _ in range(6))
    fin, fin_e = np.zeros((len(seqs), d)), np.zeros((len(seqs), d))
    for s, (lo, hi) in enumerate(seqs):
        ch = np.zeros(d) if initial is None else initial[s]
        cm, ce = np.abs(ch), np.zeros(d)
        for t in range(lo, hi):
            before[t], before_m[t], before_e[t] = ch, cm, ce
            ce = a[t] * ce + (ra[t] + 2 * U) * a[t] * cm + b_e[t]
            ch, cm = a[t] * ch + b[t], a[t] * cm + np.abs(b[t])
            ce = ce + 2 * U * cm
            h[t], m[t], e[t] = ch, cm, ce
        fin[s], fin_e[s] = ch, ce
    out = {"y": (h, e), "final": (fin, fin_e)}
    if dy is None:
        return out
    dh, md, ed = (np.zeros((rows, d)) for _ in range(3))
    ini, ini_e = np.zeros((len(seqs), d)), np.zeros((len(seqs), d))
    for s, (lo, hi) in enumerate(seqs):
        gv = np.zeros(d) if dfinal is None else dfinal[s]
        gm, ge = np.abs(gv), np.zeros(d)
        for t in range(hi - 1, lo - 1, -1):
            dh[t], md[t] = dy[t] + gv, np.abs(dy[t]) + gm
            ed[t] = ge + 2 * U * md[t]
            gv, gm = a[t] * dh[t], a[t] * md[t]
            ge = a[t] * ed[t] + (ra[t] + 2 * U) * gm
        ini[s], ini_e[s] = gv, ge
    out["dinitial"] = (ini, ini_e)
    out["dx"] = (dh * w * g, product(md, ed, w * g, (rw + rg + U) * w * g))
    other = sigmoid(-inp)  # 1 - g
    fi = w * g * x * other
    out["dinput"] = (dh * fi, product(md, ed, fi, (rw + 2 * rg + (2 * np.abs(inp) + 8) * U) * np.abs(fi)))
    slope = np.divide(f, w, out=np.zeros_like(w), where=w > 0)
    p1, p2 = a * f * before, a * a * g * x * slope
    p1_e = a * f * before_e + (ra + rf + 3 * U) * a * f * before_m
    p2_e = (2 * ra + rg + rf + rw + 6 * U) * np.abs(p2)
    fr = p1 - p2
    fr_e = p1_e + p2_e + 2 * U * (a * f * before_m + np.abs(p2))
    off = sigmoid(-decay)  # 1 - f
    fd = fr * rate * off
    fd_e = fr_e * np.abs(rate) * off + (rf + (2 * np.abs(decay) + 8) * U) * (np.abs(p1) + np.abs(p2)) * np.abs(rate) * off
    out["ddecay"] = (dh * fd, product(md, ed, fd, fd_e))
    # drate: a term's way into the sum: 8 rows of a wavefront, 8 wavefronts, a sixteenth of the tiles of 64 rows, 16 parts
    terms = product(md, ed, np.abs(p1) + np.abs(p2), fr_e) + (40 + rows / 1024) * U * md * (np.abs(p1) + np.abs(p2))
    out["drate"] = ((dh * fr).sum(0), terms.sum(0))
    return {q: (v, 1.01 * err) for q, (v, err) in out.items()}
