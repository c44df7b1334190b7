"""Error bounds of the selective scan that follow the recurrence.

``sequence_reference.scan`` counts every rounding of the longest sequence against the largest
magnitude.  Here the error of a row is carried to the next one: what a factor a = exp(dt A) < 1
forgets of the state it also forgets of the state's error,

    m[t] = a m[t-1] + |b[t]|                      (m: the state over magnitudes, b = dt x B)
    e[t] = a e[t-1] + ra a m[t-1] + rb |b[t]| + U m[t]

with ra, rb the relative errors of the factor and of the new term.  So a bound stays a small
multiple of 2^-24 however long the sequence is, and a state held in fewer bits leaves it.

Roundings counted (U = 2^-24 each; exp2, log2 and reciprocal of the hardware are good to one unit
in the last place, 2 U):
    raw = delta + bias                      1
    dt = softplus(raw)                      8, and raw's error times softplus' = sigmoid(raw)
    dt A: A log2(e) (2), the product (1);   3 times |dt A|, and |A| times dt's error
    a = exp2(..)                            2
    joined spans                            exp2(A sum dt): the sum of at most `longest` steps, so
                                            `longest` times |dt A| for each step's share
    b = dt x B                              2, and dt's
    silu(z) = z / (1 + exp2(-z log2 e))     2 |z| + 8
    sums over N states                      N + 2
First-order terms; products of errors are covered by the factor 1.01 at the end."""
import numpy as np

import sequence_reference as ref

U = ref.U


def scan(x, delta, A, B, C, D=None, z=None, bias=None, sp=True, seqs=(), initial=None, dy=None, dfinal=None):
    """{name: (value, error before the final rounding)}; arguments as sequence_reference.scan's."""
    args = (x, delta, A, B, C, D, z, bias, sp, seqs, initial, dy, dfinal)
    val = ref._scan(*args, absolute=False)
    rows, d = x.shape
    g, n = B.shape[1:]
    rep = d // g
    longest = max([hi - lo for lo, hi in seqs] + [0])
    raw = delta + (0 if bias is None else bias)
    dt = ref.softplus(raw) if sp else raw
    raw_e = U * np.abs(raw)
    dt_e = 8 * U * np.abs(dt) + ref.sigmoid(raw) * raw_e if sp else raw_e
    Aa, xa, dta = np.abs(A), np.abs(x), np.abs(dt)
    Bw, Cw = np.repeat(np.abs(B), rep, 1), np.repeat(np.abs(C), rep, 1)
    zA = dta[:, :, None] * Aa
    a = np.exp(dt[:, :, None] * A)
    ra = (3 + longest) * U * zA + Aa * dt_e[:, :, None] + 2 * U
    dx = dta * xa
    dx_e = xa * dt_e + U * dx
    b = dx[:, :, None] * Bw
    b_e = dx_e[:, :, None] * Bw + U * b
    m, e, before, before_e = (np.zeros((rows, d, n)) for _ in range(4))
    fin_e = np.zeros((len(seqs), d, n))
    for s, (lo, hi) in enumerate(seqs):
        cm = np.zeros((d, n)) if initial is None else np.abs(initial[s])
        ce = np.zeros((d, n))
        for t in range(lo, hi):
            before[t], before_e[t] = cm, ce
            ce = a[t] * ce + ra[t] * a[t] * cm + b_e[t]
            cm = a[t] * cm + b[t]
            ce += U * cm
            m[t], e[t] = cm, ce
        fin_e[s] = ce
    out = {"final": fin_e}
    Da = np.zeros(d) if D is None else np.abs(D)
    v = (Cw * m).sum(-1) + Da * xa
    v_e = (Cw * e).sum(-1) + (n + 2) * U * (Cw * m).sum(-1) + 2 * U * v
    if z is None:
        gate, gate_r = np.ones_like(x), np.zeros_like(x)
    else:
        gate, gate_r = np.abs(ref.silu(z)), (2 * np.abs(z) + 8) * U
    out["y"] = gate * (v_e + (gate_r + U) * v)
    if dy is not None:
        dya = np.abs(dy)
        dv = dya * gate
        dv_e = (gate_r + U) * dv
        md, ed = np.zeros((rows, d, n)), np.zeros((rows, d, n))
        ini_e = np.zeros((len(seqs), d, n))
        for s, (lo, hi) in enumerate(seqs):
            gm = np.zeros((d, n)) if dfinal is None else np.abs(dfinal[s])
            ge = np.zeros((d, n))
            for t in range(hi - 1, lo - 1, -1):
                md[t] = dv[t][:, None] * Cw[t] + gm
                ed[t] = ge + dv_e[t][:, None] * Cw[t] + 2 * U * md[t]
                gm = a[t] * md[t]
                ge = a[t] * ed[t] + (ra[t] + U) * gm
            ini_e[s] = ge
        out["dinitial"] = ini_e

        def product(p, pe, q, qe, roundings=1):
            return p * qe + q * pe + roundings * U * p * q

        def fold(q):
            return q.reshape(rows, g, rep, n).sum(2)
        out["dC"] = fold(product(dv[:, :, None], dv_e[:, :, None], m, e)) + (rep + 16) * U * fold(dv[:, :, None] * m)
        out["dB"] = fold(product(dx[:, :, None], dx_e[:, :, None], md, ed)) + (rep + 16) * U * fold(dx[:, :, None] * md)
        along = (md * Bw).sum(-1)
        along_e = (ed * Bw).sum(-1) + (n + 3) * U * along
        through = a * md * before
        through_e = a * (ed * before + md * before_e) + (ra + 3 * U) * through
        sd = (through * Aa).sum(-1)
        sd_e = (through_e * Aa).sum(-1) + (n + 6) * U * sd
        out["dx"] = product(dta, dt_e, along, along_e) + Da * dv_e + 2 * U * (dv * Da + dta * along)
        ddt = along * xa + sd
        ddt_e = xa * along_e + sd_e + 2 * U * ddt
        if sp:
            sg = ref.sigmoid(raw)
            # sigmoid: as silu's, and the error of raw times sigmoid' <= sigmoid
            out["ddelta"] = sg * (ddt_e + ((2 * np.abs(raw) + 8) * U + raw_e) * ddt)
            ddelta = sg * ddt
        else:
            out["ddelta"], ddelta = ddt_e, ddt
        out["dA"] = (product(dta[:, :, None], dt_e[:, :, None], through, through_e)).sum(0) + (rows + 8) * U * (dta[:, :, None] * through).sum(0)
        out["dD"] = (xa * dv_e).sum(0) + (rows + 8) * U * (xa * dv).sum(0)
        out["ddelta_bias"] = out["ddelta"].sum(0) + (rows + 8) * U * ddelta.sum(0)
        if z is not None:
            # silu' = s (1 + z (1 - s)) over magnitudes s (1 + |z|)
            slope = ref.sigmoid(z) * (1 + np.abs(z))
            out["dz"] = dya * slope * (v_e + (2 * np.abs(z) + 16) * U * v)
    return {q: (val[q], 1.01 * out[q]) for q in out}


def outside(got, want, error, half=U, tiny=2.0 ** -126):
    """Where `got` (float64 array) is further from `want` than the error and one rounding to a type of relative half step `half`."""
    return ~(np.abs(got - want) <= error + half * (np.abs(want) + error) + tiny)


def near(got, want, error, what):
    """`got` (a tensor) within the error of `want`, rounded once to its type."""
    bad = outside(ref.f64(got), want, error, ref.HALF[got.dtype], ref.TINY[got.dtype])
    assert not bad.any(), "%s: %d of %d values outside, worst by a factor of %.3g" % (
        what, bad.sum(), bad.size, (np.abs(ref.f64(got) - want) / (error + ref.HALF[got.dtype] * np.abs(want) + ref.TINY[got.dtype])).max())


# ---------------------------------------------------------------------- parameter sums of the convolution
def conv_sums(x, dy, w, bias, rows_skipped=None):
    """(dweight, dbias, their error bounds) of the silu convolution over (B, L, D) in 64 bits, the rows of
    `rows_skipped` (a slice of the flat rows) left out of the sums.

    Each element is bounded by its own terms g x.  The longest way of a term into the sum: 128 rows of a
    lane, 32 row groups of a workgroup, a quarter of the workgroups' sums (at most rows / 128 of them) and
    3 more; g itself: K + 1 roundings of u, silu' (2 |u| + 12), the product with dy."""
    b, l, d = x.shape
    k = w.shape[1]
    u = np.zeros((b, l, d)) + bias
    mu = np.abs(u)
    taps = []
    for q in range(k):
        tap = np.zeros((b, l, d))
        tap[:, k - 1 - q:] = x[:, :l - (k - 1 - q)]
        taps.append(tap)
        u += tap * w[:, q]
        mu += np.abs(tap * w[:, q])
    s = ref.sigmoid(u)
    g = dy * s * (1 + u * (1 - s))
    # |silu''| <= 1/2; the roundings of silu' are relative to s (1 + |u|)
    g_e = np.abs(dy) * ((k + 1) * U * mu / 2 + (2 * np.abs(u) + 12) * U * s * (1 + np.abs(u))) + U * np.abs(g)
    keep = np.ones(b * l)
    if rows_skipped is not None:
        keep[rows_skipped] = 0
    keep = keep.reshape(b, l, 1)
    count = (128 + 32 + b * l / 128 / 4 + 4) * U
    dw = np.stack([(keep * g * t).sum((0, 1)) for t in taps], 1)
    dw_e = np.stack([((g_e + count * np.abs(g)) * np.abs(t)).sum((0, 1)) for t in taps], 1)
    return dw, (keep * g).sum((0, 1)), 1.01 * dw_e, 1.01 * (g_e + count * np.abs(g)).sum((0, 1))
