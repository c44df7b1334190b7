"""The sequence operators on the GPU against their formulas in 64 bits (sequence_reference.py, which
also derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sequence_reference as ref
from sequence_reference import close, f64

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(rng, *shape, t=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(t).cuda()


def wider(x, rng, left=8, right=8):
    """x as a slice of a tensor with more columns, which hold NaN."""
    w = torch.full(x.shape[:-1] + (left + x.shape[-1] + right,), float("nan"), dtype=x.dtype, device=x.device)
    w[..., left:left + x.shape[-1]] = x
    return w[..., left:left + x.shape[-1]]


def offsets(lengths, first=0):
    return torch.tensor(np.cumsum([first] + list(lengths)), dtype=torch.int32, device="cuda")


def same(a, b, what):
    assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.cpu(), b.cpu()), what


# ---------------------------------------------------------------------- embedding
def lookup_reference(tokens, table, scale):
    """A product in 32 bits, rounded once: equal bit for bit."""
    tok = tokens.cpu().long()
    inside = (tok >= 0) & (tok < table.shape[0])
    rows = table.cpu().float()[tok.clamp(0, table.shape[0] - 1)] * torch.tensor(scale, dtype=torch.float32)
    return torch.where(inside[..., None], rows, torch.zeros(())).to(table.dtype)


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("n,v,d", [(0, 5, 8), (1, 1, 1), (3, 7, 5), (65, 300, 64), (130, 1000, 515), (66, 90, 590), (77, 50, 2056), (1000, 40000, 96)])
def test_lookup(t, n, v, d):
    rng = np.random.default_rng(n + d)
    for dtype in (torch.int32, torch.int64):
        tok = torch.from_numpy(rng.integers(-2, v + 2, n)).to(dtype).cuda()
        for table in (randn(rng, v, d, t=T[t]), wider(randn(rng, v, d, t=T[t]), rng)):
            same(dw.embedding_lookup(tok, table, scale=1.7), lookup_reference(tok, table, 1.7), "n=%d v=%d d=%d" % (n, v, d))


def test_lookup_shapes_and_extreme_tokens():
    rng = np.random.default_rng(1)
    table = randn(rng, 9, 24, t=torch.bfloat16)
    table[3] = float("inf")
    tok = torch.tensor([[3, 8, 0], [-(1 << 62), (1 << 62), 1 << 32]], dtype=torch.int64, device="cuda")
    y = dw.embedding_lookup(tok, table)
    assert y.shape == (2, 3, 24)
    same(y, lookup_reference(tok, table, 1.0), "extreme tokens")  # 2^32 is not token 0
    out = torch.empty_like(y)
    assert dw.embedding_lookup(tok, table, out=out) is out
    same(out, y, "out")


def grad_reference(tok, dout, v, scale):
    """(value, magnitude, count) per row"""
    t = tok.cpu().numpy().reshape(-1).astype(np.int64)
    g = f64(dout).reshape(-1, dout.shape[-1])
    val, mag = np.zeros((v, g.shape[1])), np.zeros((v, g.shape[1]))
    ok = (t >= 0) & (t < v)
    np.add.at(val, t[ok], g[ok])
    np.add.at(mag, t[ok], np.abs(g[ok]))
    count = np.bincount(t[ok], minlength=v).max() + 3 if ok.any() else 1
    return val * np.float64(np.float32(scale)), mag * scale, count


def tokens_of(kind, rng, n, v):
    if kind == "uniform":
        t = rng.integers(-1, v + 1, n)
    elif kind == "one":
        t = np.full(n, v // 2)
    elif kind == "few":  # byte-like tokens in a large table
        t = rng.integers(0, min(v, 16), n)
    elif kind == "none":
        t = np.where(rng.integers(0, 2, n) == 0, -5, v)
    else:  # falling frequencies
        t = np.minimum(np.exp(rng.uniform(0, math.log(v + 1.0), n)).astype(np.int64), v) - 1
    return torch.from_numpy(t)


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("kind", ["uniform", "one", "few", "none", "skewed"])
@pytest.mark.parametrize("n,v,d", [(0, 3, 8), (1, 1, 1), (5, 9, 3), (64, 20, 64), (65, 257, 40), (90, 300, 590),
                                   (1000, 700, 72), (4097, 3000, 17)])
def test_grad(t, kind, n, v, d):
    rng = np.random.default_rng(n + v)
    tok = tokens_of(kind, rng, n, v).int().cuda()
    dout = randn(rng, n, d, t=T[t])
    val, mag, count = grad_reference(tok, dout, v, 0.75)
    g = dw.embedding_grad(tok, dout, v, scale=0.75)
    close(g, val, mag, count, "grad %s n=%d" % (kind, n))
    same(g, dw.embedding_grad(tok.long(), wider(dout, rng), v, scale=0.75), "64-bit tokens, strided")
    g32 = dw.embedding_grad(tok, dout, v, scale=0.75, out=torch.full((v, d), float("nan"), device="cuda"))
    close(g32, val, mag, count, "float32 gradient")
    # accumulated: rows without a position keep what they hold
    base = randn(rng, v, d)
    acc = base.clone()
    dw.embedding_grad(tok, dout, v, scale=0.75, out=acc, accumulate=True)
    close(acc, val + f64(base), mag + np.abs(f64(base)), count + 1, "accumulated")
    absent = torch.ones(v, dtype=torch.bool)
    absent[tok.cpu().long()[(tok.cpu() >= 0) & (tok.cpu() < v)]] = False
    same(acc.cpu()[absent], base.cpu()[absent], "rows left alone")


@pytest.mark.parametrize("n,v,d,kind", [(65536, 100000, 8, "skewed"), (65537, 100000, 8, "skewed"), (70001, 1000, 16, "few"),
                                        (200003, 150001, 4, "uniform"), (131072, 64, 8, "one"), (3000, 600000, 8, "uniform")])
def test_grad_segments(n, v, d, kind):
    """More tokens than one pass of the grouping reads, and tables with more rows than its counters."""
    rng = np.random.default_rng(n)
    tok = tokens_of(kind, rng, n, v).int().cuda()
    dout = randn(rng, n, d)
    val, mag, count = grad_reference(tok, dout, v, 1.0)
    g = dw.embedding_grad(tok, dout, v)
    close(g, val, mag, count, "segments n=%d" % n)
    for _ in range(2):
        same(dw.embedding_grad(tok, dout, v), g, "repeats bit for bit")


# ---------------------------------------------------------------------- convolution
CONV_LENGTHS = [[1], [2, 0, 1, 7], [0, 0], [33, 64, 5], [130], [16, 16, 1, 0, 47, 3]]


def conv_check(got, want, names, what):
    for name, g in zip(names, got):
        close(g, *want[name], "%s %s" % (what, name))


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("k", [2, 3, 4])
@pytest.mark.parametrize("lengths,d", list(zip(CONV_LENGTHS, [1, 24, 8, 515, 72, 200])))
def test_conv_packed(t, k, lengths, d):
    rng = np.random.default_rng(sum(lengths) + d + k)
    rows, t = sum(lengths), T[t]
    for weight_t, act, with_state, strided in ((t, "silu", True, True), (torch.float32, None, False, False)):
        x, dy = randn(rng, rows, d, t=t), randn(rng, rows, d, t=t)
        w, b = randn(rng, d, k, t=weight_t), randn(rng, d, t=weight_t)
        init = randn(rng, len(lengths), k - 1, d, t=t) if with_state else None
        dfin = randn(rng, len(lengths), k - 1, d, t=t) if with_state else None
        bias = b if with_state else None
        if strided:
            x, dy = wider(x, rng), wider(dy, rng)
        off = offsets(lengths)
        want = ref.conv(f64(x), f64(w), f64(bias), act == "silu", ref.ranges(None, off.tolist()), f64(init), f64(dy), f64(dfin))
        y, fin = dw.causal_conv1d(x, w, bias, activation=act, seq_offsets=off, initial_state=init, final_state=True)
        conv_check((y, fin), want, ("y", "final"), "packed")
        g = dw.causal_conv1d_grad(dy, x, w, bias, activation=act, seq_offsets=off, initial_state=init, dfinal_state=dfin)
        assert (g.dbias is None) == (bias is None) and (g.dinitial_state is None) == (init is None)
        names = ("dx", "dweight") + (("dbias", "dinitial") if with_state else ())
        conv_check([v for v in g if v is not None], want, names, "packed")


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l,d", [(1, 1, 64), (3, 1, 7), (2, 37, 40), (5, 3, 136), (1, 300, 8), (2, 0, 16), (9, 70, 520)])
def test_conv_batch(t, b, l, d):
    rng = np.random.default_rng(b * l + d)
    t = T[t]
    x, dy = randn(rng, b, l, d, t=t), wider(randn(rng, b, l, d, t=t), rng)
    w, bias = randn(rng, d, 4, t=t), randn(rng, d, t=t)
    want = ref.conv(f64(x).reshape(-1, d), f64(w), f64(bias), True, ref.ranges(x.shape, None), None, f64(dy).reshape(-1, d))
    y = dw.causal_conv1d(x, w, bias, activation="silu")
    assert y.shape == x.shape
    close(y.reshape(-1, d), *want["y"], "y")
    wide = torch.full((b, l, 2 * d), 3.0, dtype=t, device="cuda")
    g = dw.causal_conv1d_grad(dy, x, w, bias, activation="silu", dx=wide[..., d:])
    conv_check((wide[..., d:].reshape(-1, d), g.dweight, g.dbias), want, ("dx", "dweight", "dbias"), "batch")
    assert (wide[..., :d] == 3.0).all()


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("rows,d,k", [(1, 1, 2), (3, 64, 4), (17, 264, 3), (70, 33, 4)])
def test_conv_step(t, rows, d, k):
    """Steps from slots in any order against the prompt form; slots outside the state are skipped."""
    rng = np.random.default_rng(rows + d)
    t = T[t]
    w, b = randn(rng, d, k, t=t), randn(rng, d, t=t)
    state = randn(rng, rows + 2, k - 1, d, t=t)
    slots = torch.from_numpy(rng.permutation(rows + 2)[:rows].astype(np.int32)).cuda()
    skipped = rows > 2
    if skipped:
        slots[1], slots[2] = -1, rows + 2
    xs = randn(rng, 5, rows, d, t=t)
    start = state.clone()
    ys = []
    for i in range(5):
        out = torch.full((rows, d), 9.0, dtype=t, device="cuda")
        ys.append(dw.causal_conv1d_step(wider(xs[i], rng), state, w, b, activation="silu", slots=slots, out=out))
    y = torch.stack(ys)
    live = [i for i in range(rows) if not (skipped and i in (1, 2))]
    seqs = [(5 * q, 5 * q + 5) for q in range(len(live))]
    x = f64(xs)[:, live].transpose(1, 0, 2).reshape(-1, d)
    want = ref.conv(x, f64(w), f64(b), True, seqs, f64(start)[slots.cpu().numpy()[live]])
    close(y[:, live].transpose(0, 1).reshape(-1, d), *want["y"], "y")
    same(state[slots[live].long()], torch.from_numpy(want["final"][0]).to(t), "state")
    if skipped:
        assert (y[:, 1:3] == 9.0).all()
    untouched = [s for s in range(rows + 2) if s not in set(slots.cpu().numpy()[live].tolist())]
    same(state[untouched], start[untouched], "other slots")


def test_conv_rows_outside_the_sequences():
    """Rows before the first offset and behind the last one hold NaN: neither read nor written."""
    rng = np.random.default_rng(3)
    d, k, lengths = 40, 4, [5, 0, 9]
    x = torch.full((20, d), float("nan"), device="cuda")
    x[2:16] = randn(rng, 14, d)
    off = offsets(lengths, 2)
    w, b = randn(rng, d, k), randn(rng, d)
    dy = torch.full((20, d), float("nan"), device="cuda")
    dy[2:16] = randn(rng, 14, d)
    want = ref.conv(f64(x)[2:16], f64(w), f64(b), False, [(0, 5), (5, 5), (5, 14)], None, f64(dy)[2:16])
    out = torch.full((20, d), 4.0, device="cuda")
    y = dw.causal_conv1d(x, w, b, seq_offsets=off, out=out)
    close(y[2:16], *want["y"], "y")
    dx = torch.full((20, d), 4.0, device="cuda")
    g = dw.causal_conv1d_grad(dy, x, w, b, seq_offsets=off, dx=dx)
    close(dx[2:16], *want["dx"], "dx")
    close(g.dweight, *want["dweight"], "dweight")
    for v in (y, dx):
        assert (v[:2] == 4.0).all() and (v[16:] == 4.0).all()


# ---------------------------------------------------------------------- scan
def scan_inputs(rng, lead, d, n, g, t, strided):
    lead = tuple(lead)
    v = dict(x=randn(rng, *lead, d, t=t), delta=randn(rng, *lead, d, t=t), z=randn(rng, *lead, d, t=t),
             B=randn(rng, *lead, g, n, t=t), C=randn(rng, *lead, g, n, t=t))
    if strided:
        for q in ("x", "delta", "z"):
            v[q] = wider(v[q], rng)
        both = torch.cat([v["B"].flatten(-2), v["C"].flatten(-2)], -1)
        v["B"], v["C"] = (both[..., :g * n].unflatten(-1, (g, n)), both[..., g * n:].unflatten(-1, (g, n)))
    v["A"] = -torch.from_numpy(rng.uniform(0.2, 3.0, (d, n))).float().cuda()
    v["D"] = randn(rng, d)
    v["delta_bias"] = randn(rng, d) - 2.0
    return v


def scan_reference(v, seqs, initial=None, dy=None, dfinal=None, sp=True):
    d, (g, n) = v["x"].shape[-1], v["B"].shape[-2:]
    flat = lambda q, *s: f64(v[q]).reshape(-1, *s) if v.get(q) is not None else None  # noqa: E731
    return ref.scan(flat("x", d), flat("delta", d), f64(v["A"]), flat("B", g, n), flat("C", g, n), f64(v.get("D")), flat("z", d),
                    f64(v.get("delta_bias")), sp, seqs, f64(initial), None if dy is None else f64(dy).reshape(-1, d), f64(dfinal))


def call_args(v):
    return (v["x"], v["delta"], v["A"], v["B"], v["C"]), {k: v[k] for k in ("D", "z", "delta_bias") if v.get(k) is not None}


def scan_check(got, want, what):
    for name, g in got.items():
        val = want[name]
        close(g.reshape(val[0].shape), *val, "%s %s" % (what, name))


def grads_dict(g):
    r = {k: v for k, v in g._asdict().items() if v is not None}
    if "dinitial_state" in r:
        r["dinitial"] = r.pop("dinitial_state")
    return r


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("lengths,d,n,g", [([1], 1, 1, 1), ([2, 0, 31, 1], 24, 16, 2), ([0, 0], 16, 16, 1), ([33, 64, 5], 80, 16, 1),
                                           ([130], 136, 13, 2), ([16, 17, 1, 0, 47, 3], 66, 16, 3), ([70, 9], 40, 32, 1),
                                           ([45, 0, 50], 24, 64, 2), ([20, 33], 10, 40, 1), ([300, 2, 211], 24, 16, 1)])
def test_scan_packed(t, lengths, d, n, g):
    rng = np.random.default_rng(sum(lengths) + d + n)
    rows, t = sum(lengths), T[t]
    off = offsets(lengths)
    seqs = ref.ranges(None, off.tolist())
    for full in (True, False):
        v = scan_inputs(rng, (rows,), d, n, g, t, strided=full)
        init = randn(rng, len(lengths), d, n) if full else None
        dfin = randn(rng, len(lengths), d, n) if full else None
        if not full:
            v["D"] = v["z"] = v["delta_bias"] = None
            v["delta"] = v["delta"].abs() * 0.3
        dy = wider(randn(rng, rows, d, t=t), rng) if full else randn(rng, rows, d, t=t)
        want = scan_reference(v, seqs, init, dy, dfin, sp=full)
        a, kw = call_args(v)
        kw.update(delta_softplus=full, seq_offsets=off, initial_state=init)
        y, fin, saved = dw.selective_scan(*a, final_state=True, save_for_grad=True, **kw)
        scan_check(dict(y=y, final=fin), want, "packed")
        grads = dw.selective_scan_grad(dy, *a, saved=saved, dfinal_state=dfin, **kw)
        scan_check(grads_dict(grads), want, "packed")
        assert (grads.dD is None) == (grads.dz is None) == (grads.ddelta_bias is None) == (not full)
        again = dw.selective_scan_grad(dy, *a, dfinal_state=dfin, **kw)  # the states scanned again
        for p, q in zip(grads, again):
            assert (p is None and q is None) or torch.equal(p, q), "repeats bit for bit"


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l,d,n,g", [(1, 1, 16, 16, 1), (3, 1, 7, 5, 1), (2, 37, 40, 16, 1), (5, 3, 132, 16, 2), (1, 700, 16, 16, 1),
                                       (2, 0, 16, 16, 1), (3, 290, 64, 16, 4), (2, 260, 20, 33, 1), (40, 33, 192, 16, 1)])
def test_scan_batch(t, b, l, d, n, g):
    rng = np.random.default_rng(b * l + d + n)
    t = T[t]
    v = scan_inputs(rng, (b, l), d, n, g, t, strided=True)
    dy = randn(rng, b, l, d, t=t)
    seqs = ref.ranges(v["x"].shape, None)
    init, dfin = randn(rng, b, d, n), randn(rng, b, d, n)
    want = scan_reference(v, seqs, init, dy, dfin)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, initial_state=init)
    fin = torch.full((b, d, n), float("nan"), device="cuda")
    y, same_fin, saved = dw.selective_scan(*a, final_state=fin, save_for_grad=True, **kw)
    assert same_fin is fin and y.shape == v["x"].shape
    scan_check(dict(y=y, final=fin), want, "batch")
    both = torch.full((b, l, 2 * d), 3.0, dtype=t, device="cuda")
    grads = dw.selective_scan_grad(dy, *a, saved=saved, dfinal_state=dfin, dx=both[..., :d], dz=both[..., d:], **kw)
    scan_check(grads_dict(grads), want, "batch")


@pytest.mark.parametrize("d", [16, 200])
def test_scan_many_short_sequences(d):
    """Hundreds of sequences of no row to a few (a batch of drafts, say): several in every span, spans that
    begin and end inside them."""
    rng = np.random.default_rng(40 + d)
    lengths = [int(v) for v in rng.integers(0, 6, 300)] + [70] + [0, 0, 1]
    rows, n = sum(lengths), 16
    v = scan_inputs(rng, (rows,), d, n, 1, torch.float32, strided=False)
    off = offsets(lengths)
    init, dfin, dy = randn(rng, len(lengths), d, n), randn(rng, len(lengths), d, n), randn(rng, rows, d)
    want = scan_reference(v, ref.ranges(None, off.tolist()), init, dy, dfin)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=off, initial_state=init)
    y, fin, saved = dw.selective_scan(*a, final_state=True, save_for_grad=True, **kw)
    scan_check(dict(y=y, final=fin), want, "many")
    scan_check(grads_dict(dw.selective_scan_grad(dy, *a, saved=saved, dfinal_state=dfin, **kw)), want, "many")


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("rows,d,n,g", [(1, 1, 1, 1), (3, 64, 16, 2), (9, 40, 64, 1), (17, 70, 9, 2), (5, 24, 32, 3)])
def test_scan_step(t, rows, d, n, g):
    """Steps from slots in any order against the recurrence; slots outside the state are skipped."""
    rng = np.random.default_rng(rows + d)
    t = T[t]
    steps = 4
    v = scan_inputs(rng, (steps, rows), d, n, g, t, strided=True)
    state = randn(rng, rows + 2, d, n)
    start = state.clone()
    slots = torch.from_numpy(rng.permutation(rows + 2)[:rows].astype(np.int32)).cuda()
    skipped = rows > 2
    if skipped:
        slots[0], slots[2] = -7, rows + 2
    y = torch.full((steps, rows, d), 9.0, dtype=t, device="cuda")
    for i in range(steps):
        dw.selective_scan_step(v["x"][i], v["delta"][i], v["A"], v["B"][i], v["C"][i], state, D=v["D"], z=v["z"][i],
                               delta_bias=v["delta_bias"], delta_softplus=True, slots=slots, out=y[i])
    live = [i for i in range(rows) if not (skipped and i in (0, 2))]
    seqs = [(steps * q, steps * q + steps) for q in range(len(live))]
    w = {k: (q.cpu()[:, live].transpose(0, 1).contiguous() if q.dim() > 2 else q) for k, q in v.items() if k not in ("A",)}
    w["A"] = v["A"]
    want = scan_reference(w, seqs, start[slots[live].long()])
    close(y[:, live].transpose(0, 1).reshape(-1, d), *want["y"], "y")
    close(state[slots[live].long()], *want["final"], "state")
    if skipped:
        assert (y[:, [0, 2]] == 9.0).all()
    untouched = [s for s in range(rows + 2) if s not in set(slots.cpu().numpy()[live].tolist())]
    same(state[untouched], start[untouched], "other slots")


def test_scan_rows_outside_the_sequences():
    rng = np.random.default_rng(8)
    d, n, rows, lo, hi = 72, 16, 300, 3, 280
    lengths = [100, 0, 177]
    v = scan_inputs(rng, (rows,), d, n, 1, torch.float32, strided=False)
    dy = randn(rng, rows, d)
    for q in ("x", "delta", "z", "B", "C"):
        v[q][:lo], v[q][hi:] = float("nan"), float("inf")
    dy[:lo], dy[hi:] = float("nan"), float("nan")
    off = offsets(lengths, lo)
    inner = {k: (q[lo:hi] if q.shape[0] == rows else q) for k, q in v.items()}
    want = scan_reference(inner, [(0, 100), (100, 100), (100, 277)], None, dy[lo:hi], None)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=off)
    out = torch.full((rows, d), 4.0, device="cuda")
    y, fin, saved = dw.selective_scan(*a, final_state=True, save_for_grad=True, out=out, **kw)
    scan_check(dict(y=y[lo:hi], final=fin), want, "inner rows")
    dx = torch.full((rows, d), 4.0, device="cuda")
    g = dw.selective_scan_grad(dy, *a, saved=saved, dx=dx, **kw)
    scan_check(dict(dx=dx[lo:hi], dB=g.dB[lo:hi], dC=g.dC[lo:hi], dA=g.dA, dD=g.dD, ddelta_bias=g.ddelta_bias,
                    dz=g.dz[lo:hi], ddelta=g.ddelta[lo:hi]), want, "inner rows")
    for q in (out, dx):
        assert (q[:lo] == 4.0).all() and (q[hi:] == 4.0).all()


def test_scan_large_steps_and_extreme_values():
    """Steps beyond softplus's threshold, a state that is forgotten at once, and gates that saturate."""
    rng = np.random.default_rng(9)
    rows, d, n = 50, 16, 16
    v = scan_inputs(rng, (rows,), d, n, 1, torch.float32, strided=False)
    v["delta"][::7] = 40.0
    v["delta"][3::7] = -60.0
    v["z"][::5] = 200.0
    v["z"][1::5] = -200.0
    dy = randn(rng, rows, d)
    want = scan_reference(v, [(0, rows)], None, dy)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=offsets([rows]))
    scan_check(dict(y=dw.selective_scan(*a, **kw)), want, "extremes")
    scan_check(grads_dict(dw.selective_scan_grad(dy, *a, **kw)), want, "extremes")


def test_scan_not_a_number_stays_in_its_channel_and_sequence():
    rng = np.random.default_rng(10)
    d, n = 48, 16
    v = scan_inputs(rng, (60,), d, n, 1, torch.float32, strided=False)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=offsets([20, 40]))
    clean = dw.selective_scan(*a, **kw)
    v["x"][5, 7] = float("nan")
    y = dw.selective_scan(*a, **kw)
    hit = torch.zeros(60, d, dtype=torch.bool, device="cuda")
    hit[5:20, 7] = True
    assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])


def test_linear_gradients_match_differences():
    """y is linear in x, B, C and D one at a time: its change along a direction is the gradient's product
    with it, up to the roundings of the two outputs (the reference's bound on y, summed over y's weights)."""
    rng = np.random.default_rng(12)
    v = scan_inputs(rng, (90,), 40, 16, 2, torch.float32, strided=False)
    dy = randn(rng, 90, 40)
    kw = dict(delta_softplus=True, seq_offsets=offsets([50, 40]), z=v["z"], delta_bias=v["delta_bias"])
    names = ("x", "delta", "A", "B", "C")

    def run(u):
        return f64(dw.selective_scan(*[u[k] for k in names], D=u["D"], **kw))
    g = dw.selective_scan_grad(dy, *[v[k] for k in names], D=v["D"], **kw)
    want = scan_reference(v, [(0, 50), (50, 90)], None, dy)
    for name, grad in (("x", g.dx), ("B", g.dB), ("C", g.dC), ("D", g.dD)):
        step = randn(rng, *v[name].shape)
        up, down = dict(v), dict(v)
        up[name], down[name] = v[name] + step, v[name] - step
        got = ((run(up) - run(down)) / 2 * f64(dy)).sum()
        exact_step = (f64(up[name]) - f64(down[name])) / 2
        bound = 0.0
        for u in (up, down):
            r = scan_reference(u, [(0, 50), (50, 90)])["y"]
            bound += ((r[2] * ref.U * r[1] + 2 ** -24 * np.abs(r[0])) * np.abs(f64(dy))).sum() / 2
        q = {"x": "dx", "B": "dB", "C": "dC", "D": "dD"}[name]
        bound += ((want[q][2] + 1) * ref.U * want[q][1] * np.abs(exact_step)).sum()
        assert abs(got - (f64(grad) * exact_step).sum()) <= bound, name


# ---------------------------------------------------------------------- sizes that take the other shapes
@pytest.mark.parametrize("t,n", [("bf16", 16), ("f32", 5)])
def test_scan_step_many_rows(t, n):
    """Enough rows that a wavefront takes four of them, with slots that end inside such a four."""
    rng = np.random.default_rng(30 + n)
    rows, d, t = 2051, 130, T[t]
    v = scan_inputs(rng, (1, rows), d, n, 1, t, strided=True)
    state = randn(rng, rows, d, n)
    start = state.clone()
    slots = torch.from_numpy(rng.permutation(rows).astype(np.int32)).cuda()
    slots[::97] = -1
    y = torch.full((rows, d), 9.0, dtype=t, device="cuda")
    dw.selective_scan_step(v["x"][0], v["delta"][0], v["A"], v["B"][0], v["C"][0], state, D=v["D"], z=v["z"][0],
                           delta_bias=v["delta_bias"], delta_softplus=True, slots=slots, out=y)
    live = (slots >= 0).nonzero()[:, 0]
    w = {k: (q[:, live] if q.dim() > 2 else q) for k, q in v.items()}
    at = slots[live].long()
    want = scan_reference(w, [(i, i + 1) for i in range(live.numel())], start[at])
    close(y[live], *want["y"], "y")
    close(state[at], *want["final"], "state")
    assert (y[slots < 0] == 9.0).all()
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[at] = False
    same(state[rest], start[rest], "other slots")


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_conv_long_blocks_match_short_ones(t):
    """64 sequences at once take the longest row blocks, one at a time shorter ones: the same bits per
    row; the weights' sums within their bound."""
    rng = np.random.default_rng(31)
    b, l, d, t = 64, 700, 1024, T[t]
    x, dy = randn(rng, b, l, d, t=t), randn(rng, b, l, d, t=t)
    w, bias = randn(rng, d, 4, t=t), randn(rng, d, t=t)
    y = dw.causal_conv1d(x, w, bias, activation="silu")
    g = dw.causal_conv1d_grad(dy, x, w, bias, activation="silu")
    dweight, dbias, mag = torch.zeros(d, 4, dtype=torch.float64), torch.zeros(d, dtype=torch.float64), 0.0
    for i in range(b):
        yi = dw.causal_conv1d(x[i:i + 1], w, bias, activation="silu")
        gi = dw.causal_conv1d_grad(dy[i:i + 1], x[i:i + 1], w, bias, activation="silu")
        assert torch.equal(yi[0], y[i]) and torch.equal(gi.dx[0], g.dx[i])
        dweight += gi.dweight.double().cpu()
        dbias += gi.dbias.double().cpu()
    # |act'| <= 1.1: the terms of a sum over rows are at most 1.1 |dy| |x|; two sums of b l terms each
    largest = 1.1 * float((dy.abs().amax() * torch.clamp(x.abs().amax(), min=1.0)).float())
    bound = 2 * b * l * 2 ** -24 * b * l * largest
    assert (g.dweight.double().cpu() - dweight).abs().max() <= bound and (g.dbias.double().cpu() - dbias).abs().max() <= bound


def test_offsets_past_32_bits():
    """Rows, slots and table rows whose element offsets pass 2^31."""
    rng = np.random.default_rng(32)
    rows, tail, d, n = 540001, 150, 64, 16
    big = torch.zeros(rows, 4096, dtype=torch.bfloat16, device="cuda")  # 2.2e9 elements
    assert rows * 4096 > 2 ** 31
    v = scan_inputs(rng, (tail,), d, n, 1, torch.bfloat16, strided=False)
    x = big[:, 64:64 + d]
    x[-tail:] = v["x"]
    off = torch.tensor([0, rows - tail, rows], dtype=torch.int32, device="cuda")
    w, b = randn(rng, d, 4, t=torch.bfloat16), randn(rng, d, t=torch.bfloat16)
    want = ref.conv(f64(v["x"]), f64(w), f64(b), True, [(0, tail)], None, f64(v["x"]))
    close(dw.causal_conv1d(x, w, b, activation="silu", seq_offsets=off)[-tail:], *want["y"], "conv y")
    close(dw.causal_conv1d_grad(x, x, w, b, activation="silu", seq_offsets=off).dx[-tail:], *want["dx"], "conv dx")
    z = big[:, 256:256 + d]
    z[-tail:] = v["z"]
    bc = big[:, 512:512 + 2 * n]
    bc[-tail:, :n], bc[-tail:, n:] = v["B"].flatten(-2), v["C"].flatten(-2)
    B, C = bc[:, :n].unflatten(-1, (1, n)), bc[:, n:].unflatten(-1, (1, n))
    v["delta"] = v["x"]
    want = scan_reference(v, [(0, tail)], None, v["z"])
    kw = dict(D=v["D"], z=z, delta_bias=v["delta_bias"], delta_softplus=True, seq_offsets=off)
    y, saved = dw.selective_scan(x, x, v["A"], B, C, save_for_grad=True, **kw)
    close(y[-tail:], *want["y"], "scan y")
    g = dw.selective_scan_grad(z, x, x, v["A"], B, C, saved=saved, **kw)
    scan_check(dict(dx=g.dx[-tail:], dz=g.dz[-tail:], dB=g.dB[-tail:], dC=g.dC[-tail:]), want, "past 32 bits")
    # tables and states
    tok = torch.tensor([rows - 1, 7, rows - 2], dtype=torch.int32, device="cuda")
    same(dw.embedding_lookup(tok, big), big[tok.long()], "lookup")
    gt = dw.embedding_grad(tok, big[-3:], rows)
    same(gt[tok.long()], big[-3:], "table gradient")
    del big, gt, x, z, bc, B, C, g, y
    slots = 33000
    state = torch.zeros(slots, 4096, n, device="cuda")  # 2.2e9 elements
    one = scan_inputs(rng, (1, 2), 4096, n, 1, torch.float32, strided=False)
    at = torch.tensor([slots - 1, 5], dtype=torch.int32, device="cuda")
    state[at.long()] = randn(rng, 2, 4096, n)
    start = state[at.long()]
    y = dw.selective_scan_step(one["x"][0], one["delta"][0], one["A"], one["B"][0], one["C"][0], state, D=one["D"], z=one["z"][0],
                               delta_bias=one["delta_bias"], delta_softplus=True, slots=at)
    want = scan_reference(one, [(0, 1), (1, 2)], start)
    close(y, *want["y"], "step y")
    close(state[at.long()], *want["final"], "step state")


def test_scan_infinite_input_without_skip():
    """Without D there is no term of it: an infinite x reaches y through the state alone."""
    d, n = 16, 16
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    x = one(1, 3, d)
    x[0, 1, 4] = float("inf")
    args = (x, one(1, 3, d), -one(d, n), one(1, 3, 1, n), one(1, 3, 1, n))
    y = dw.selective_scan(*args)
    state = torch.zeros(1, d, n, device="cuda")
    steps = [dw.selective_scan_step(x[:, i], args[1][:, i], args[2], args[3][:, i], args[4][:, i], state) for i in range(3)]
    for v in (y[0], torch.cat(steps)):
        assert (v[1:, 4] == float("inf")).all() and torch.isfinite(v[:, :4]).all() and torch.isfinite(v[0]).all()


# ---------------------------------------------------------------------- together, graphs, streams
def block(p, tokens, off=None, conv_state=None, scan_state=None):
    """Embedding, convolution, scan: a prompt."""
    e = dw.embedding_lookup(tokens, p["table"], scale=2.0)
    u, cs = dw.causal_conv1d(e, p["w"], p["b"], activation="silu", seq_offsets=off, initial_state=conv_state, final_state=True)
    bc = u[..., :2 * p["g"] * p["n"]].unflatten(-1, (2 * p["g"], p["n"]))
    y, ss = dw.selective_scan(u, e, p["A"], bc[..., :p["g"], :], bc[..., p["g"]:, :], D=p["D"], z=e, delta_bias=p["db"],
                              delta_softplus=True, seq_offsets=off, initial_state=scan_state, final_state=True)
    return y, cs, ss


def params(rng, v=500, d=72, n=16, g=2, t=torch.float32):
    return dict(table=randn(rng, v, d, t=t, scale=0.5), w=randn(rng, d, 4, t=t), b=randn(rng, d, t=t), g=g, n=n, d=d, v=v,
                A=-torch.from_numpy(rng.uniform(0.2, 3.0, (d, n))).float().cuda(), D=randn(rng, d), db=randn(rng, d) - 2.0)


def test_prompt_equals_its_pieces_and_single_tokens():
    """Packed prompts in one call, the same prompts in two calls that pass their states on, and token
    by token from slots: the operators' results for float32, within the prompt's own error bound."""
    rng = np.random.default_rng(20)
    p = params(rng)
    lengths = [40, 1, 170]
    tok = torch.from_numpy(rng.integers(0, p["v"], sum(lengths)).astype(np.int32)).cuda()
    off = offsets(lengths)
    y, cs, ss = block(p, tok, off)
    # in two pieces
    cut = [13, 0, 101]
    first = torch.cat([tok[o:o + c] for o, c in zip(off.tolist(), cut)])
    rest = torch.cat([tok[o + c:o + n] for o, c, n in zip(off.tolist(), cut, lengths)])
    y1, cs1, ss1 = block(p, first, offsets(cut))
    y2, cs2, ss2 = block(p, rest, offsets([n - c for n, c in zip(lengths, cut)]), cs1, ss1)
    same(cs2, cs, "convolution state")
    # token by token
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cstate, sstate = torch.zeros(5, 3, p["d"], device="cuda"), torch.zeros(5, p["d"], p["n"], device="cuda")
    steps = torch.zeros_like(y)
    o = off.tolist()
    for t in range(max(lengths)):
        live = [s for s in range(3) if t < lengths[s]]
        at = torch.tensor([o[s] + t for s in live], device="cuda")
        e = dw.embedding_lookup(tok[at], p["table"], scale=2.0)
        u = dw.causal_conv1d_step(e, cstate, p["w"], p["b"], activation="silu", slots=slots[live])
        bc = u[:, :2 * p["g"] * p["n"]].unflatten(-1, (2 * p["g"], p["n"]))
        steps[at] = dw.selective_scan_step(u, e, p["A"], bc[:, :p["g"]], bc[:, p["g"]:], sstate, D=p["D"], z=e, delta_bias=p["db"],
                                           delta_softplus=True, slots=slots[live])
    same(cstate[slots.long()], cs, "convolution state, token by token")
    # the bound: every form is within it of the 64-bit scan of the convolution's output
    e = dw.embedding_lookup(tok, p["table"], scale=2.0)
    u = dw.causal_conv1d(e, p["w"], p["b"], activation="silu", seq_offsets=off)
    bc = u[:, :2 * p["g"] * p["n"]].unflatten(-1, (2 * p["g"], p["n"]))
    v = dict(x=u, delta=e, A=p["A"], B=bc[:, :p["g"]], C=bc[:, p["g"]:], D=p["D"], z=e, delta_bias=p["db"])
    want = scan_reference(v, ref.ranges(None, o))
    scan_check(dict(y=y, final=ss), want, "prompt")
    pieces = torch.zeros_like(y)
    o1, o2 = 0, 0
    for s in range(3):
        c, m = cut[s], lengths[s] - cut[s]
        pieces[o[s]:o[s] + c], pieces[o[s] + c:o[s + 1]] = y1[o1:o1 + c], y2[o2:o2 + m]
        o1, o2 = o1 + c, o2 + m
    scan_check(dict(y=pieces, final=ss2), want, "pieces")
    scan_check(dict(y=steps, final=sstate[slots.long()]), want, "steps")


def train_pass(p, tok, dy):
    """Forward and backward of the block by hand (B and C of their own, so that gradients do not meet)."""
    e = dw.embedding_lookup(tok, p["table"], scale=2.0)
    u = dw.causal_conv1d(e, p["w"], p["b"], activation="silu")
    y, saved = dw.selective_scan(u, p["delta"], p["A"], p["B"], p["C"], D=p["D"], delta_bias=p["db"], delta_softplus=True, save_for_grad=True)
    s = dw.selective_scan_grad(dy, u, p["delta"], p["A"], p["B"], p["C"], D=p["D"], delta_bias=p["db"], delta_softplus=True, saved=saved)
    c = dw.causal_conv1d_grad(s.dx, e, p["w"], p["b"], activation="silu")
    return [y, dw.embedding_grad(tok, c.dx, p["v"], scale=2.0), c.dweight, c.dbias] + [q for q in s if q is not None]


def train_params(rng, b=2, l=300, **kw):
    p = params(rng, **kw)
    t = p["table"].dtype
    p.update(delta=randn(rng, b, l, p["d"], t=t), B=randn(rng, b, l, p["g"], p["n"], t=t), C=randn(rng, b, l, p["g"], p["n"], t=t))
    tok = torch.from_numpy(rng.integers(-1, p["v"], (b, l)).astype(np.int32)).cuda()
    return p, tok, randn(rng, b, l, p["d"], t=t)


def test_training_chain_matches_autograd_of_the_formulas():
    """The chain's gradients against torch.autograd in 64 bits on the host, relative to the largest value
    of each: 300 rows of a recurrence and the sums over them stay below 2^-24 * 300 * 32."""
    rng = np.random.default_rng(21)
    p, tok, dy = train_params(rng)
    got = train_pass(p, tok, dy)
    leaf = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items() if torch.is_tensor(v)}
    tk = tok.cpu().long()
    e = torch.where((tk >= 0)[..., None], leaf["table"][tk.clamp(min=0)] * 2.0, 0.0)
    u = torch.nn.functional.pad(e, (0, 0, 3, 0)).unfold(1, 4, 1).mul(leaf["w"]).sum(-1) + leaf["b"]
    u = torch.nn.functional.silu(u)
    dt = torch.nn.functional.softplus(leaf["delta"] + leaf["db"])
    per = p["d"] // p["g"]
    h, ys = torch.zeros(2, p["d"], p["n"], dtype=torch.float64), []
    for i in range(u.shape[1]):
        h = torch.exp(dt[:, i, :, None] * leaf["A"]) * h + (dt[:, i] * u[:, i])[..., None] * leaf["B"][:, i].repeat_interleave(per, 1)
        ys.append((h * leaf["C"][:, i].repeat_interleave(per, 1)).sum(-1) + leaf["D"] * u[:, i])
    y = torch.stack(ys, 1)
    names = ("table", "w", "b")
    grads = torch.autograd.grad(y, [leaf[k] for k in names + ("delta", "A", "B", "C", "D", "db")], dy.double().cpu())
    want = [y.detach()] + list(grads[:3]) + [None] + list(grads[3:])
    for g, w in zip(got, want):
        if w is not None:
            assert g.shape == w.shape
            assert (g.double().cpu() - w).abs().max() <= 2 ** -24 * 300 * 32 * w.abs().max()


def test_graphs_replay_with_workspaces_of_their_own():
    """Two captured training passes, replayed by turns and on two streams at once with eager work between."""
    rng = np.random.default_rng(22)
    sets = [train_params(rng), train_params(rng, d=40)]
    eager = [train_pass(*s) for s in sets]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for s in sets:
            train_pass(*s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(train_pass(*s))
            graphs.append(g)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for turn in range(3):
        for g, o in zip(graphs, outs):
            for q in o:
                q.fill_(7.0)
        torch.cuda.synchronize()
        if turn == 1:
            graphs[0].replay()
            train_pass(*sets[1])
            graphs[1].replay()
        else:
            with torch.cuda.stream(side):
                graphs[0].replay()
            with torch.cuda.stream(other):
                graphs[1].replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            for q, w in zip(o, e):
                assert torch.equal(q, w)


def test_streams():
    """A stream object or a raw handle, the call's memory coming from that stream."""
    rng = np.random.default_rng(23)
    p, tok, dy = train_params(rng, l=64)
    u = randn(rng, 2, 64, p["d"])
    want = dw.selective_scan(u, p["delta"], p["A"], p["B"], p["C"], delta_softplus=True)
    conv = dw.causal_conv1d(u, p["w"], p["b"])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        y = dw.selective_scan(u, p["delta"], p["A"], p["B"], p["C"], delta_softplus=True, stream=stream)
        c = dw.causal_conv1d(u, p["w"], p["b"], stream=stream)
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(c, conv)


def test_device_refusals():
    rng = np.random.default_rng(24)
    x, w = randn(rng, 2, 6, 16), randn(rng, 16, 4)
    A, bc = randn(rng, 16, 16), randn(rng, 2, 6, 1, 16)
    for bad in (lambda: dw.causal_conv1d(x, w.cpu()), lambda: dw.causal_conv1d(x[0], w), lambda: dw.causal_conv1d(x, w, activation="gelu"),
                lambda: dw.causal_conv1d(x, w[:8]), lambda: dw.causal_conv1d(x.transpose(0, 1), w),
                lambda: dw.causal_conv1d(x, w, out=x), lambda: dw.causal_conv1d(x, w, initial_state=x),
                lambda: dw.causal_conv1d(x[0], w, seq_offsets=offsets([6]).long()),
                lambda: dw.causal_conv1d(x, randn(rng, 16, 5)), lambda: dw.causal_conv1d(x, w.half()),
                lambda: dw.selective_scan(x, x, A.half(), bc, bc), lambda: dw.selective_scan(x, x.half(), A, bc, bc),
                lambda: dw.selective_scan(x, x, A, bc, bc[:, :5]), lambda: dw.selective_scan(x, x, A, bc.expand(2, 6, 3, 16), bc),
                lambda: dw.selective_scan(x, x, A, bc, bc, D=x), lambda: dw.selective_scan(x, x, A, bc, bc, out=x),
                lambda: dw.selective_scan_grad(x, x, x, A, bc, bc, saved=A), lambda: dw.selective_scan_grad(x, x, x, A, bc, bc, dz=x),
                lambda: dw.selective_scan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], randn(rng, 1, 16, 16)),
                lambda: dw.embedding_lookup(torch.zeros(3, device="cuda"), w), lambda: dw.embedding_lookup(torch.zeros(3, dtype=torch.int32), w),
                lambda: dw.embedding_grad(torch.zeros(2, 6, dtype=torch.int32, device="cuda"), x, 5, accumulate=True),
                lambda: dw.embedding_grad(torch.zeros(6, dtype=torch.int32, device="cuda"), x, 5),
                lambda: dw.embedding_grad(torch.zeros(2, 6, dtype=torch.int32, device="cuda"), x, 0)):
        with pytest.raises((TypeError, ValueError, dw.ScanError)):
            bad()
    # nothing above reached the GPU
    assert torch.isfinite(dw.causal_conv1d(x, w)).all()
