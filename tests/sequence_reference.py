"""The sequence operators from their formulas, in 64 bits on the host, row by row.

Each function also bounds the error that 32-bit arithmetic in any order of summation may make:
it runs the same formulas over magnitudes (every term replaced by its absolute value, so that
nothing cancels) and counts the roundings on the longest way into a result.  A result of type t
may then differ from the 64-bit one by

    eps(t) / 2 * |value|  +  count * 2^-24 * magnitude

where the first term is the final rounding and the second every rounding before it.  An
exponential's argument z with relative error r gives a factor with relative error |z| r, so a step
of the recurrence h' = exp(dt A) h + ... costs 3 roundings (the exponential's own, the product,
the sum) and |dt A| times those of dt (softplus: at most 8) and of the product (2).
"""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(got, want, magnitude, count, what):
    """`got` (a tensor) within the bound of `want`; values below the type's normal range may flush to zero."""
    t = got.dtype
    g = f64(got)
    assert g.shape == want.shape, (what, g.shape, want.shape)
    tol = HALF[t] * (np.abs(want) + count * U * magnitude) + count * U * magnitude + TINY[t]
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        k = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / tol, 0)), g.shape)
        raise AssertionError("%s: %d of %d values differ, worst at %s: %r instead of %r (tolerance %r)"
                             % (what, bad.sum(), bad.size, k, g[k], want[k], tol[k]))


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def ranges(x_shape, seq_offsets):
    """The sequences' row ranges."""
    if seq_offsets is not None:
        o = [int(v) for v in seq_offsets]
        return list(zip(o[:-1], o[1:]))
    return [(s * x_shape[1], (s + 1) * x_shape[1]) for s in range(x_shape[0])]


# ---------------------------------------------------------------------- convolution
def conv(x, w, b, act, seqs, initial, dy=None, dfinal=None):
    """x (rows, D), w (D, K), initial (S, K-1, D) or None.  Returns {name: (value, magnitude, count)}."""
    rows, d = x.shape
    k = w.shape[1]
    fill = np.zeros
    u, mu = fill((rows, d)), fill((rows, d))
    fin = fill((len(seqs), k - 1, d))
    whole = {}
    for s, (lo, hi) in enumerate(seqs):
        first = np.zeros((k - 1, d)) if initial is None else initial[s]
        whole[s] = np.concatenate([first, x[lo:hi]])
        fin[s] = whole[s][hi - lo:]
        for t in range(lo, hi):
            taps = whole[s][t - lo:t - lo + k]
            u[t] = (taps * w.T).sum(0) + (0 if b is None else b)
            mu[t] = (np.abs(taps) * np.abs(w.T)).sum(0) + (0 if b is None else np.abs(b))
    y = silu(u) if act else u
    # |silu'| < 1.1; the activation's own roundings are relative to |u|
    out = {"y": (y, 1.1 * mu + np.abs(u), k + 10), "final": (fin, np.abs(fin), 0)}
    if dy is None:
        return out
    da = dsilu(u) if act else np.ones_like(u)
    g = dy * da
    mg = np.abs(dy) * (1.0 + mu if act else 1.0)  # |silu''| <= 1/2
    n = {q: np.zeros(sh) for q, sh in (("dx", (rows, d)), ("dweight", (d, k)), ("dbias", (d,)), ("dinitial", (len(seqs), k - 1, d)))}
    m = {q: np.zeros_like(v) for q, v in n.items()}
    for s, (lo, hi) in enumerate(seqs):
        dw_, mw_ = np.zeros_like(whole[s]), np.zeros_like(whole[s])
        for t in range(lo, hi):
            sl = slice(t - lo, t - lo + k)
            dw_[sl] += g[t] * w.T
            mw_[sl] += mg[t] * np.abs(w.T)
            n["dweight"] += (g[t] * whole[s][sl]).T
            m["dweight"] += (mg[t] * np.abs(whole[s][sl])).T
            n["dbias"] += g[t]
            m["dbias"] += mg[t]
        if dfinal is not None:
            dw_[hi - lo:] += dfinal[s]
            mw_[hi - lo:] += np.abs(dfinal[s])
        n["dx"][lo:hi], m["dx"][lo:hi] = dw_[k - 1:], mw_[k - 1:]
        n["dinitial"][s], m["dinitial"][s] = dw_[:k - 1], mw_[:k - 1]
    for q in n:
        out[q] = (n[q], m[q], 2 * k + 16 + (rows if q in ("dweight", "dbias") else 0))
    return out


# ---------------------------------------------------------------------- scan
def softplus(v):
    return np.logaddexp(v, 0.0)


def _scan(x, delta, A, B, C, D, z, bias, sp, seqs, initial, dy, dfinal, absolute):
    """The recurrence and its adjoint.  With `absolute`, over magnitudes."""
    m = np.abs if absolute else (lambda v: v)
    rows, d = x.shape
    g, n = B.shape[1:]
    rep = d // g
    raw = delta + (0 if bias is None else bias)
    dt = softplus(raw) if sp else raw
    a = np.exp(dt[:, :, None] * A)  # positive either way
    xa, Aa, dta = m(x), m(A), m(dt)
    Bw, Cw = np.repeat(m(B), rep, 1), np.repeat(m(C), rep, 1)
    Da = np.zeros(d) if D is None else m(D)
    h, before = np.zeros((rows, d, n)), np.zeros((rows, d, n))
    out = {"final": np.zeros((len(seqs), d, n))}
    for s, (lo, hi) in enumerate(seqs):
        cur = np.zeros((d, n)) if initial is None else m(initial[s])
        for t in range(lo, hi):
            before[t] = cur
            cur = a[t] * cur + (dta[t] * xa[t])[:, None] * Bw[t]
            h[t] = cur
        out["final"][s] = cur
    v = (h * Cw).sum(-1) + Da * xa
    gate = np.ones_like(x) if z is None else m(silu(z))
    out["y"] = v * gate
    if dy is None:
        return out
    dya = m(dy)
    dv = dya * gate
    dh = np.zeros((rows, d, n))
    out["dinitial"] = np.zeros((len(seqs), d, n))
    for s, (lo, hi) in enumerate(seqs):
        cur = np.zeros((d, n)) if dfinal is None else m(dfinal[s])
        for t in range(hi - 1, lo - 1, -1):
            dh[t] = dv[t][:, None] * Cw[t] + cur
            cur = a[t] * dh[t]
        out["dinitial"][s] = cur
    if z is not None:
        # silu' lies between 0.1 below 0 and 1.1; the error of the gate's slope is relative to its terms
        out["dz"] = dya * v * (1.0 + np.abs(z) if absolute else dsilu(z))
    fold = lambda q: q.reshape(rows, g, rep, n).sum(2)  # noqa: E731
    out["dC"] = fold(dv[:, :, None] * h)
    out["dB"] = fold(dh * (dta * xa)[:, :, None])
    along = (dh * Bw).sum(-1)
    through = dh * a * before
    out["dx"] = dv * Da + dta * along
    ddt = along * xa + (through * Aa).sum(-1)
    out["ddelta"] = ddt * sigmoid(raw) if sp else ddt
    out["dA"] = (through * dta[:, :, None]).sum(0)
    out["dD"] = (dv * xa).sum(0)
    out["ddelta_bias"] = out["ddelta"].sum(0)
    return out


def scan(x, delta, A, B, C, D=None, z=None, bias=None, sp=False, seqs=(), initial=None, dy=None, dfinal=None):
    """{name: (value, magnitude, count)}; x, delta, z, dy (rows, D), B, C (rows, G, N)."""
    args = (x, delta, A, B, C, D, z, bias, sp, seqs, initial, dy, dfinal)
    val, mag = _scan(*args, absolute=False), _scan(*args, absolute=True)
    raw = delta + (0 if bias is None else bias)
    dt = softplus(raw) if sp else raw
    zmax = float(np.abs(dt[:, :, None] * A).max()) if x.shape[0] else 0.0
    longest = max([hi - lo for lo, hi in seqs] + [0])
    # 8 roundings of dt, 2 of the product, in units of |dt A|; 4 per step; the gate and the rest: 32
    steps = longest * (4 + 10 * zmax) + A.shape[1] + 32 + 10 * zmax
    rows, d = x.shape
    extra = {"dA": rows, "dD": rows, "ddelta_bias": rows, "dB": d, "dC": d}
    out = {}
    for q in val:
        back = q.startswith("d")
        out[q] = (val[q], mag[q], (2 if back else 1) * steps + extra.get(q, 0) + (0 if not back else 32))
    return out
