"""The gated linear recurrence on the GPU against its formulas in 64 bits (gated_reference.py, which also derives
the error bounds)."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import gated_reference as gr
import sequence_reference as ref
from sequence_errors import near
from sequence_reference import f64

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


def inputs(rng, lead, d, t, strided=False):
    """x, both gates, rates from strong to hardly any decay."""
    v = [randn(rng, *lead, d, t=t, scale=s) for s in (1.0, 2.0, 2.0)]
    if strided:
        v = [wider(q, rng) for q in v]
    return v + [-torch.from_numpy(np.exp(rng.uniform(np.log(1e-3), np.log(8.0), d))).float().cuda()]


def reference(v, seqs, initial=None, dy=None, dfinal=None):
    d = v[0].shape[-1]
    flat = [f64(q).reshape(-1, d) for q in v[:3]]
    return gr.gated(*flat, f64(v[3]), seqs, f64(initial), None if dy is None else f64(dy).reshape(-1, d), f64(dfinal))


def check(got, want, what):
    for name, g in got.items():
        near(g.reshape(want[name][0].shape), *want[name], "%s %s" % (what, name))


def named(g):
    r = dict(dx=g.dx, ddecay=g.ddecay_gate, dinput=g.dinput_gate, drate=g.drate)
    if g.dinitial_state is not None:
        r["dinitial"] = g.dinitial_state
    return r


# 64 rows to a tile, 8 tiles to a group
LENGTHS = [[1], [2, 0, 31, 1], [0, 0], [64], [65], [33, 64, 5], [128, 0, 64], [130], [7, 120, 1, 0, 47, 300], [1024], [1025, 3],
           [5, 2200], [640, 640, 1100]]


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("lengths,d", list(zip(LENGTHS, [1, 24, 8, 300, 515, 72, 200, 258, 66, 5, 64, 12, 7])))
def test_packed(t, lengths, d):
    rng = np.random.default_rng(sum(lengths) + d)
    rows, t = sum(lengths), T[t]
    off = offsets(lengths)
    seqs = ref.ranges(None, off.tolist())
    for full in (True, False):
        v = inputs(rng, (rows,), d, t, strided=full)
        init = randn(rng, len(lengths), d) if full else None
        dfin = randn(rng, len(lengths), d) if full else None
        dy = wider(randn(rng, rows, d, t=t), rng) if full else randn(rng, rows, d, t=t)
        want = reference(v, seqs, init, dy, dfin)
        kw = dict(seq_offsets=off, initial_state=init)
        y, fin, saved = dw.gated_scan(*v, final_state=True, save_for_grad=True, **kw)
        check(dict(y=y, final=fin), want, "packed")
        g = dw.gated_scan_grad(dy, *v, saved=saved, dfinal_state=dfin, **kw)
        check(named(g), want, "packed")
        assert (g.dinitial_state is None) == (not full)
        again = dw.gated_scan_grad(dy, *v, dfinal_state=dfin, **kw)  # the states scanned again
        for p, q in zip(g, again):
            assert (p is None and q is None) or torch.equal(p, q), "repeats bit for bit"


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l,d", [(1, 1, 16), (3, 1, 7), (2, 37, 40), (5, 3, 132), (1, 700, 16), (2, 0, 16), (3, 290, 64), (2, 64, 260),
                                   (40, 33, 192), (70, 2, 10), (2, 1100, 6)])
def test_batch(t, b, l, d):
    rng = np.random.default_rng(b * l + d)
    t = T[t]
    v = inputs(rng, (b, l), d, t, strided=True)
    dy, init, dfin = randn(rng, b, l, d, t=t), randn(rng, b, d), randn(rng, b, d)
    want = reference(v, ref.ranges(v[0].shape, None), init, dy, dfin)
    fin = torch.full((b, d), float("nan"), device="cuda")
    y, same_fin, saved = dw.gated_scan(*v, initial_state=init, final_state=fin, save_for_grad=True)
    assert same_fin is fin and y.shape == v[0].shape
    check(dict(y=y, final=fin), want, "batch")
    wide = torch.full((b, l, 3 * d), 3.0, dtype=t, device="cuda")
    g = dw.gated_scan_grad(dy, *v, initial_state=init, dfinal_state=dfin, saved=saved, dx=wide[..., :d], ddecay_gate=wide[..., d:2 * d])
    check(named(g), want, "batch")
    assert (wide[..., 2 * d:] == 3.0).all()
    out = torch.full((b, l, d + 5), 3.0, dtype=t, device="cuda")
    dw.gated_scan(*v, initial_state=init, out=out[..., :d])
    assert torch.equal(out[..., :d], y) and (out[..., d:] == 3.0).all()


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l,d", [(260, 130, 24), (128, 65, 200), (33, 200, 1030), (256, 128, 3), (130, 65, 128), (100, 70, 140)])
def test_many_sequences_at_once(t, b, l, d):
    """Enough sequences that workgroups walk through whole ones in the gradient; last tiles of one to all rows."""
    rng = np.random.default_rng(b + l + d)
    t = T[t]
    v = inputs(rng, (b, l), d, t, strided=True)
    dy, init, dfin = randn(rng, b, l, d, t=t), randn(rng, b, d), randn(rng, b, d)
    want = reference(v, ref.ranges(v[0].shape, None), init, dy, dfin)
    y, fin, saved = dw.gated_scan(*v, initial_state=init, final_state=True, save_for_grad=True)
    check(dict(y=y, final=fin), want, "many")
    g = dw.gated_scan_grad(dy, *v, initial_state=init, dfinal_state=dfin, saved=saved)
    check(named(g), want, "many")
    bare = reference(v, ref.ranges(v[0].shape, None), None, dy)
    check(named(dw.gated_scan_grad(dy, *v)), bare, "many, no states")
    for p, q in zip(g, dw.gated_scan_grad(dy, *v, initial_state=init, dfinal_state=dfin, saved=saved)):
        assert torch.equal(p, q)


def test_many_short_sequences():
    rng = np.random.default_rng(41)
    lengths = [int(v) for v in rng.integers(0, 6, 900)] + [170] + [0, 0, 1]
    rows, d = sum(lengths), 40
    v = inputs(rng, (rows,), d, torch.float32)
    init, dfin, dy = randn(rng, len(lengths), d), randn(rng, len(lengths), d), randn(rng, rows, d)
    off = offsets(lengths)
    want = reference(v, ref.ranges(None, off.tolist()), init, dy, dfin)
    y, fin, saved = dw.gated_scan(*v, seq_offsets=off, initial_state=init, final_state=True, save_for_grad=True)
    check(dict(y=y, final=fin), want, "many")
    check(named(dw.gated_scan_grad(dy, *v, seq_offsets=off, initial_state=init, dfinal_state=dfin, saved=saved)), want, "many")


@pytest.mark.parametrize("t,lengths,d", [("bf16", [20000], 512), ("f32", [9000, 1, 0, 11000], 130), ("f16", [5000] * 4, 255)])
def test_long_sequences(t, lengths, d):
    """Hundreds of tiles in a chain: within the bounds in some channels, and bit for bit the same every time."""
    rng = np.random.default_rng(42 + d)
    rows, t = sum(lengths), T[t]
    v = inputs(rng, (rows,), d, t)
    init, dfin, dy = randn(rng, len(lengths), d), randn(rng, len(lengths), d), randn(rng, rows, d, t=t)
    off = offsets(lengths)
    kw = dict(seq_offsets=off, initial_state=init)
    y, fin, saved = dw.gated_scan(*v, final_state=True, save_for_grad=True, **kw)
    g = dw.gated_scan_grad(dy, *v, saved=saved, dfinal_state=dfin, **kw)
    some = torch.tensor([0, 1, 63, 64, 127, d // 2, d - 2, d - 1], device="cuda")
    pick = lambda q: q[:, some] if q.dim() == 2 else q[some]  # noqa: E731
    want = reference([pick(q) for q in v], ref.ranges(None, off.tolist()), pick(init), pick(dy), pick(dfin))
    check({k: pick(q) for k, q in dict(named(g), y=y, final=fin).items()}, want, "long")
    for _ in range(4):
        y2, fin2, saved2 = dw.gated_scan(*v, final_state=True, save_for_grad=True, **kw)
        g2 = dw.gated_scan_grad(dy, *v, saved=saved2, dfinal_state=dfin, **kw)
        for p, q in zip((y, fin) + tuple(g), (y2, fin2) + tuple(g2)):
            assert torch.equal(p, q)


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 64), (17, 264), (70, 33), (5, 2054), (600, 130)])
def test_step(t, rows, d):
    """Steps from slots in any order against the recurrence; slots outside the state are skipped."""
    rng = np.random.default_rng(rows + d)
    t, steps = T[t], 4
    v = inputs(rng, (steps, rows), d, t, strided=True)
    state = randn(rng, rows + 2, d)
    start = state.clone()
    slots = torch.from_numpy(rng.permutation(rows + 2)[:rows].astype(np.int32)).cuda()
    skipped = [0, 2] if rows > 2 else []
    for q, s in zip(skipped, (-7, rows + 2)):
        slots[q] = s
    y = torch.full((steps, rows, d), 9.0, dtype=t, device="cuda")
    for i in range(steps):
        dw.gated_scan_step(v[0][i], v[1][i], v[2][i], v[3], state, slots=slots, out=y[i])
    live = [i for i in range(rows) if i not in skipped]
    seqs = [(steps * q, steps * q + steps) for q in range(len(live))]
    want = reference([q.cpu()[:, live].transpose(0, 1) for q in v[:3]] + [v[3]], seqs, start[slots[live].long()])
    check(dict(y=y[:, live].transpose(0, 1), final=state[slots[live].long()]), want, "step")
    if skipped:
        assert (y[:, skipped] == 9.0).all()
    untouched = [s for s in range(rows + 2) if s not in set(slots.cpu().numpy()[live].tolist())]
    assert torch.equal(state[untouched], start[untouched])


def test_step_slots_are_rows_without_slots():
    rng = np.random.default_rng(43)
    v = inputs(rng, (6,), 20, torch.float32)
    a, b = randn(rng, 8, 20), None
    b = a.clone()
    y = dw.gated_scan_step(*v, a)
    z = dw.gated_scan_step(*v, b, slots=torch.arange(6, dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b) and torch.equal(y, z)


def test_rows_outside_the_sequences():
    """Rows before the first offset and behind the last one hold NaN: neither read nor written; new gradients are
    zero there."""
    rng = np.random.default_rng(44)
    d, rows, lo, hi = 70, 400, 67, 331
    lengths = [100, 0, 164]
    v = inputs(rng, (rows,), d, torch.float32)
    dy = randn(rng, rows, d)
    for q in v[:3] + [dy]:
        q[:lo], q[hi:] = float("nan"), float("inf")
    off = offsets(lengths, lo)
    want = reference([q[lo:hi] for q in v[:3]] + [v[3]], [(0, 100), (100, 100), (100, 264)], None, dy[lo:hi])
    out, dx = torch.full((rows, d), 4.0, device="cuda"), torch.full((rows, d), 4.0, device="cuda")
    y, fin, saved = dw.gated_scan(*v, seq_offsets=off, final_state=True, save_for_grad=True, out=out)
    g = dw.gated_scan_grad(dy, *v, seq_offsets=off, saved=saved, dx=dx)
    check(dict(y=y[lo:hi], final=fin, dx=dx[lo:hi], ddecay=g.ddecay_gate[lo:hi], dinput=g.dinput_gate[lo:hi], drate=g.drate), want, "inner")
    for q, outside in ((out, 4.0), (dx, 4.0), (g.ddecay_gate, 0.0), (g.dinput_gate, 0.0)):
        assert (q[:lo] == outside).all() and (q[hi:] == outside).all()


def test_offsets_out_of_order_stay_inside():
    """Offsets that descend or lie outside the rows give unspecified results, but nothing outside the arrays is
    written."""
    rng = np.random.default_rng(45)
    rows, d = 300, 64
    v = inputs(rng, (rows,), d, torch.float32)
    big = torch.full((3 * rows, d), 5.0, device="cuda")
    for off in ([200, 10, 290, -5, 1000], [400, 300, 200, 100, 0], [0, 299, 1, 299, 300], [-9, -9, -9, -9, -9]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        fin = torch.full((12, d), 5.0, device="cuda")
        y, _, saved = dw.gated_scan(*v, seq_offsets=off, initial_state=v[0][:4], out=big[rows:2 * rows], final_state=fin[4:8], save_for_grad=True)
        dw.gated_scan_grad(v[1], *v, seq_offsets=off, initial_state=v[0][:4], saved=saved, dx=big[rows:2 * rows])
        assert (big[:rows] == 5.0).all() and (big[2 * rows:] == 5.0).all() and (fin[:4] == 5.0).all() and (fin[8:] == 5.0).all()


def test_no_rows_and_no_sequences():
    d = 8
    z = torch.zeros(0, d, device="cuda")
    rate = -torch.ones(d, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    init = torch.arange(2.0 * d, device="cuda").view(2, d)
    y, fin = dw.gated_scan(z, z, z, rate, seq_offsets=off, initial_state=init, final_state=True)
    assert y.shape == (0, d) and torch.equal(fin, init)
    g = dw.gated_scan_grad(z, z, z, z, rate, seq_offsets=off, initial_state=init, dfinal_state=2 * init)
    assert torch.equal(g.dinitial_state, 2 * init) and (g.drate == 0).all()
    x = torch.full((70, d), float("nan"), device="cuda")
    out = torch.full((70, d), 3.0, device="cuda")
    dw.gated_scan(x, x, x, rate, seq_offsets=off[:1], out=out)
    g = dw.gated_scan_grad(x, x, x, x, rate, seq_offsets=off[:1])
    assert (out == 3.0).all() and (g.drate == 0).all() and (g.dx == 0).all()


def test_saturated_gates_and_extreme_rates():
    rng = np.random.default_rng(46)
    rows, d = 150, 24
    v = inputs(rng, (rows,), d, torch.float32)
    v[1][::7], v[1][3::7], v[1][5::11] = 60.0, -60.0, -20.0
    v[2][::5], v[2][1::5] = 200.0, -200.0
    v[3][:6] = torch.tensor([-1e-7, -0.49, -0.51, -60.0, -200.0, -1e4])
    dy, init = randn(rng, rows, d), randn(rng, 1, d)
    off = offsets([rows])
    want = reference(v, [(0, rows)], init, dy)
    y = dw.gated_scan(*v, seq_offsets=off, initial_state=init)
    check(dict(y=y), want, "extremes")
    check(named(dw.gated_scan_grad(dy, *v, seq_offsets=off, initial_state=init)), want, "extremes")


def test_no_decay_keeps_the_state():
    """Rate 0, or a decay gate of minus infinity or the type's lowest value: the state stays, x does not enter, and
    every gradient is finite."""
    rng = np.random.default_rng(47)
    rows, d = 130, 16
    for t in T.values():
        for gate in (None, float("-inf"), torch.finfo(t).min):
            v = inputs(rng, (rows,), d, t)
            if gate is None:
                v[3].zero_()
            else:
                v[1].fill_(gate)
            init, dy = randn(rng, 1, d), randn(rng, rows, d, t=t)
            off = offsets([rows])
            y = dw.gated_scan(*v, seq_offsets=off, initial_state=init)
            assert torch.equal(y, init.to(t).expand(rows, d))
            g = dw.gated_scan_grad(dy, *v, seq_offsets=off, initial_state=init)
            assert all(torch.isfinite(q).all() for q in g)
            assert (g.dx == 0).all() and (g.ddecay_gate == 0).all()


def test_not_a_number_stays_in_its_channel_and_sequence():
    rng = np.random.default_rng(48)
    d, rows = 48, 400
    v = inputs(rng, (rows,), d, torch.float32)
    off, dy = offsets([200, 200]), randn(rng, rows, d)
    clean, saved = dw.gated_scan(*v, seq_offsets=off, save_for_grad=True)
    clean_g = dw.gated_scan_grad(dy, *v, seq_offsets=off, saved=saved)
    for bad in (float("nan"), float("inf")):
        w = [q.clone() for q in v]
        w[0][50, 7] = bad
        y, saved = dw.gated_scan(*w, seq_offsets=off, save_for_grad=True)
        hit = torch.zeros(rows, d, dtype=torch.bool, device="cuda")
        hit[50:200, 7] = True
        assert not torch.isfinite(y[hit][:20]).any() and torch.equal(y[~hit], clean[~hit])
        g = dw.gated_scan_grad(dy, *w, seq_offsets=off, saved=saved)
        assert torch.equal(g.dx, clean_g.dx)  # linear in x
        for p, q in ((g.ddecay_gate, clean_g.ddecay_gate), (g.dinput_gate, clean_g.dinput_gate)):
            assert torch.equal(p[~hit], q[~hit])
        other = torch.arange(d, device="cuda") != 7
        assert torch.equal(g.drate[other], clean_g.drate[other]) and not torch.isfinite(g.drate[7])
        e = dy.clone()
        e[320, 9] = bad
        g = dw.gated_scan_grad(e, *v, seq_offsets=off)
        hit = torch.zeros(rows, d, dtype=torch.bool, device="cuda")
        hit[200:321, 9] = True
        for p, q in zip(g[:3], clean_g[:3]):
            assert torch.equal(p[~hit], q[~hit])


def test_gradients_match_differences():
    """y is linear in x and in the initial state: its change along a direction is the gradient's product with it, up
    to the two outputs' own errors."""
    rng = np.random.default_rng(49)
    rows, d = 300, 20
    v = inputs(rng, (rows,), d, torch.float32)
    off, init, dy = offsets([170, 130]), randn(rng, 2, d), randn(rng, rows, d)
    g = dw.gated_scan_grad(dy, *v, seq_offsets=off, initial_state=init)
    seqs = [(0, 170), (170, 300)]
    want = reference(v, seqs, init, dy)
    for q, grad, name in ((0, g.dx, "dx"), (4, g.dinitial_state, "dinitial")):
        args = v + [init]
        step = randn(rng, *args[q].shape)
        up, down = list(args), list(args)
        up[q], down[q] = args[q] + step, args[q] - step
        run = lambda a: f64(dw.gated_scan(*a[:4], seq_offsets=off, initial_state=a[4]))  # noqa: E731
        got = ((run(up) - run(down)) / 2 * f64(dy)).sum()
        exact = (f64(up[q]) - f64(down[q])) / 2
        bound = ((want[name][1] + gr.U * np.abs(want[name][0])) * np.abs(exact)).sum()
        for a in (up, down):
            val, err = reference(a[:4], seqs, a[4])["y"]
            bound += ((err + gr.U * np.abs(val)) * np.abs(f64(dy))).sum() / 2
        assert abs(got - (f64(grad) * exact).sum()) <= bound, name


def test_pieces_and_single_tokens_give_the_prompt():
    rng = np.random.default_rng(50)
    rows, d = 210, 36
    v = inputs(rng, (rows,), d, torch.float32)
    init = randn(rng, 1, d)
    want = reference(v, [(0, rows)], init)
    state, ys = init, []
    for lo, hi in ((0, 70), (70, 70), (70, 71), (71, 210)):
        y, state = dw.gated_scan(*[q[lo:hi] for q in v[:3]], v[3], seq_offsets=offsets([hi - lo]), initial_state=state, final_state=True)
        ys.append(y)
    check(dict(y=torch.cat(ys), final=state), want, "pieces")
    state = init.clone()
    ys = [dw.gated_scan_step(*[q[i:i + 1] for q in v[:3]], v[3], state) for i in range(rows)]
    check(dict(y=torch.cat(ys), final=state), want, "steps")


def test_offsets_past_32_bits():
    rng = np.random.default_rng(51)
    rows, tail, d = 540001, 150, 64
    big = torch.zeros(rows, 4096, dtype=torch.bfloat16, device="cuda")  # 2.2e9 elements
    parts = [big[:, 64 * i:64 * i + d] for i in range(5)]
    v = inputs(rng, (tail,), d, torch.bfloat16)
    dy = randn(rng, tail, d, t=torch.bfloat16)
    for p, q in zip(parts, v[:3] + [dy]):
        p[-tail:] = q
    off = torch.tensor([0, rows - tail, rows], dtype=torch.int32, device="cuda")
    want = reference(v, [(0, tail)], None, dy)
    y, saved = dw.gated_scan(*parts[:3], v[3], seq_offsets=off, save_for_grad=True, out=parts[4])
    check(dict(y=y[-tail:]), want, "past 32 bits")
    g = dw.gated_scan_grad(parts[3], *parts[:3], v[3], seq_offsets=off, saved=saved, dx=parts[4])
    check(dict(dx=g.dx[-tail:], ddecay=g.ddecay_gate[-tail:], dinput=g.dinput_gate[-tail:]), want, "past 32 bits")
    del big, parts, y, g
    slots = 530000
    state = torch.zeros(slots, 4096, device="cuda")  # 2.2e9 elements
    one = inputs(rng, (2,), 4096, torch.float32)
    at = torch.tensor([slots - 1, 5], dtype=torch.int32, device="cuda")
    state[at.long()] = randn(rng, 2, 4096)
    start = state[at.long()]
    y = dw.gated_scan_step(*one, state, slots=at)
    check(dict(y=y, final=state[at.long()]), reference(one, [(0, 1), (1, 2)], start), "slots past 32 bits")


def test_graphs_streams_and_overlapping_calls():
    """Captured passes with workspaces of their own, replayed by turns and at once on two streams, with eager calls
    between; a stream object and a raw handle."""
    rng = np.random.default_rng(52)
    sets = []
    for b, l, d in ((2, 1500, 72), (1, 4000, 130)):
        v = inputs(rng, (b, l), d, torch.bfloat16)
        sets.append((v, randn(rng, b, l, d, t=torch.bfloat16)))

    def run(v, dy, **kw):
        y, saved = dw.gated_scan(*v, save_for_grad=True, **kw)
        return (y,) + tuple(q for q in dw.gated_scan_grad(dy, *v, saved=saved, **kw) if q is not None)
    eager = [run(*s) for s in sets]
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for s in sets:
            run(*s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(run(*s))
            graphs.append(g)
    torch.cuda.synchronize()
    for turn in range(4):
        for o in outs:
            for q in o:
                q.fill_(7.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        if turn % 2:
            run(*sets[1])
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert all(torch.equal(p, q) for p, q in zip(o, e))
    # two calls at once, and handles
    got = []
    for stream in (side, other.cuda_stream):
        got.append(run(*sets[0], stream=stream))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(p, q) for p, q in zip(o, eager[0]))


def test_refusals():
    rng = np.random.default_rng(53)
    x = randn(rng, 2, 6, 16)
    rate = -torch.ones(16, device="cuda")
    state = torch.zeros(4, 16, device="cuda")
    for bad in (lambda: dw.gated_scan(x, x, x, rate.cpu()), lambda: dw.gated_scan(x[0], x[0], x[0], rate), lambda: dw.gated_scan(x, x, x.half(), rate),
                lambda: dw.gated_scan(x, x, x, rate[:8]), lambda: dw.gated_scan(x, x, x, rate.half()), lambda: dw.gated_scan(x, x[:, :5], x, rate),
                lambda: dw.gated_scan(x.transpose(1, 2), x, x, rate), lambda: dw.gated_scan(x, x, x, rate, out=x),
                lambda: dw.gated_scan(x, x, x, rate, initial_state=state), lambda: dw.gated_scan(x, x, x, rate, final_state=state),
                lambda: dw.gated_scan(x[0], x[0], x[0], rate, seq_offsets=offsets([6]).long()),
                lambda: dw.gated_scan_grad(x, x, x, x, rate, saved=state), lambda: dw.gated_scan_grad(x[:, :3], x, x, x, rate),
                lambda: dw.gated_scan_grad(x, x, x, x, rate, dx=x), lambda: dw.gated_scan_step(x[0], x[0], x[0], rate, state),
                lambda: dw.gated_scan_step(x[0], x[0], x[0], rate, state.half(), slots=torch.arange(6, dtype=torch.int32, device="cuda")),
                lambda: dw.gated_scan_step(x[0], x[0], x[0], rate, torch.zeros(8, 16, device="cuda"), out=x[0]),
                lambda: dw.gated_scan(x, x, x, rate.clone().requires_grad_())):
        with pytest.raises((TypeError, ValueError, dw.ScanError)):
            bad()
    assert torch.isfinite(dw.gated_scan(x, x, x, rate)).all()
