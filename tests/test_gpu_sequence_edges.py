"""The sequence operators at their edges: offsets in any order, values that are not finite, rows and
states that do not exist, sizes past a launch's limits.  Tolerances as in sequence_reference.py."""
import ctypes

import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sequence_errors as err
import sequence_reference as ref
from device_wide_prefix_tile_amd import sequence as seq
from sequence_reference import f64

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(rng, *shape, t=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(t).cuda()


def offsets(lengths, first=0):
    return torch.tensor(np.cumsum([first] + list(lengths)), dtype=torch.int32, device="cuda")


def scan_inputs(rng, lead, d, n, g=1, t=torch.float32):
    v = dict(x=randn(rng, *lead, d, t=t), delta=randn(rng, *lead, d, t=t), z=randn(rng, *lead, d, t=t),
             B=randn(rng, *lead, g, n, t=t), C=randn(rng, *lead, g, n, t=t), D=randn(rng, d), delta_bias=randn(rng, d) - 2.0)
    v["A"] = -torch.from_numpy(rng.uniform(0.2, 3.0, (d, n))).float().cuda()
    return v


def call_args(v):
    return (v["x"], v["delta"], v["A"], v["B"], v["C"]), {k: v[k] for k in ("D", "z", "delta_bias") if v.get(k) is not None}


class Bands:
    """Memory with 64 KB of a known pattern on both sides of every piece."""
    BAND = 1 << 16

    def __init__(self):
        self.all = []

    def take(self, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        size = (n + 255) // 256 * 256
        raw = torch.full((size + 2 * self.BAND,), 0xA5, dtype=torch.uint8, device="cuda")
        self.all.append((raw, n))
        return raw[self.BAND:self.BAND + n].view(dtype).view(shape)

    def check(self):
        for raw, n in self.all:
            assert (raw[:self.BAND] == 0xA5).all() and (raw[self.BAND + n:] == 0xA5).all()


# ---------------------------------------------------------------------- offsets
UNORDERED = [[0, 100, 50, 200], [0, 20, 10, 200], [200, 0, 200, 0, 130], [64, 32, 128, 0, 200], [-5, 90, 400, 30, 200],
             [-(1 << 31), (1 << 31) - 1, 3, (1 << 31) - 1], [199, 199, 7, 7, 1000], [0, 200, 0, 200, 0]]


@pytest.mark.parametrize("off", UNORDERED)
@pytest.mark.parametrize("d", [16, 200])
def test_offsets_in_any_order_stay_inside_the_arrays(off, d):
    """Offsets that descend or lie outside the rows: results are unspecified, the bytes around every output,
    saved state and workspace are not.  (tests/test_scan_walk_model.py has the same for the indices read.)"""
    rng = np.random.default_rng(len(off) + d)
    rows, n, k, seqs = 200, 16, 4, len(off) - 1
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    v = scan_inputs(rng, (rows,), d, n)
    dy, init, dfin = randn(rng, rows, d), randn(rng, seqs, d, n), randn(rng, seqs, d, n)
    good = offsets([70, 130])
    args, kw = call_args(v)
    before = dw.selective_scan(*args, delta_softplus=True, seq_offsets=good, **kw)
    mem, L = Bands(), seq._lib()

    def call(*shape, dtype=torch.float32):
        return mem.take(shape, dtype).data_ptr()
    a, _ = seq._scan_args(*args, v["D"], v["z"], v["delta_bias"], True, off, init)
    a.y, a.y_stride, a.final_state = call(rows, d), d, call(seqs, d, n)
    a.saved = call(L.selective_scan_saved(ctypes.byref(a)))
    a.workspace_bytes = L.selective_scan_workspace(ctypes.byref(a))
    a.workspace = call(a.workspace_bytes, dtype=torch.uint8)
    stream = torch.cuda.current_stream().cuda_stream
    assert L.selective_scan(ctypes.byref(a), stream) == 0
    g = seq._ScanGradArgs(a, dy.data_ptr(), d, dfin.data_ptr(), call(rows, d), d, call(rows, d), d, call(rows, d), d,
                          call(rows, n), n, call(rows, n), n, call(d, n), call(d), call(d), call(seqs, d, n))
    g.args.workspace_bytes = L.selective_scan_grad_workspace(ctypes.byref(g))
    g.args.workspace = call(g.args.workspace_bytes, dtype=torch.uint8)
    assert L.selective_scan_grad(ctypes.byref(g), stream) == 0
    w, b, cinit, cfin = randn(rng, d, k), randn(rng, d), randn(rng, seqs, k - 1, d), randn(rng, seqs, k - 1, d)
    dw.causal_conv1d(v["x"], w, b, activation="silu", seq_offsets=off, initial_state=cinit,
                     final_state=mem.take((seqs, k - 1, d), torch.float32), out=mem.take((rows, d), torch.float32))
    dw.causal_conv1d_grad(dy, v["x"], w, b, activation="silu", seq_offsets=off, initial_state=cinit, dfinal_state=cfin,
                          dx=mem.take((rows, d), torch.float32))
    torch.cuda.synchronize()
    mem.check()
    assert torch.equal(dw.selective_scan(*args, delta_softplus=True, seq_offsets=good, **kw), before)


# ---------------------------------------------------------------------- values that are not finite
def scan_values(v, lengths, dy=None, initial=None, dfinal=None, sp=True):
    """{name: value} of the formulas in 64 bits, infinities and NaN included.  The reference multiplies by a
    zero D where there is none; 2^-1000 changes no finite value and keeps infinities what they are."""
    d, (g, n) = v["x"].shape[-1], v["B"].shape[-2:]
    ends = np.cumsum([0] + list(lengths))
    with np.errstate(all="ignore"):
        r = ref.scan(f64(v["x"]), f64(v["delta"]), f64(v["A"]), f64(v["B"]), f64(v["C"]),
                     np.full(d, 2.0 ** -1000) if v.get("D") is None else f64(v["D"]), f64(v.get("z")), f64(v.get("delta_bias")), sp,
                     list(zip(ends[:-1], ends[1:])), f64(initial), None if dy is None else f64(dy), f64(dfinal))
    return {k: q[0] for k, q in r.items()}


def run_scan(v, lengths, dy, sp=True, **kw):
    a, more = call_args(v)
    kw.update(more, delta_softplus=sp, seq_offsets=offsets(lengths))
    y, fin = dw.selective_scan(*a, final_state=True, **kw)
    g = dw.selective_scan_grad(dy, *a, **kw)
    out = {k: q for k, q in g._asdict().items() if q is not None}
    if "dinitial_state" in out:
        out["dinitial"] = out.pop("dinitial_state")
    return dict(out, y=y, final=fin)


def same_where_finite(got, clean, want, want_clean, what):
    """Finite exactly where the formulas are, and the same bits as without the value wherever the formulas
    give the same (an infinite step forgets the state: what was passed back to it changes, and is finite)."""
    for name, q in got.items():
        finite = torch.from_numpy(np.isfinite(want[name])).view(q.shape)
        assert torch.equal(torch.isfinite(q).cpu(), finite), "%s %s: finite elsewhere" % (what, name)
        still = torch.from_numpy(want[name] == want_clean[name]).view(q.shape)
        assert torch.equal(q.cpu()[still], clean[name].cpu()[still]), "%s %s: other values changed" % (what, name)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["x", "delta", "z", "dy"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [16, 32, 64])
def test_scan_gradients_keep_a_row_to_itself(t, where, value, n):
    """One value that is not finite reaches what the formulas let it reach: of dB and dC, the rows of
    its own term alone, not their neighbours."""
    rng = np.random.default_rng(60 + n)
    lengths, d, t0, c0 = [40, 20], 48, 21, 37
    v = scan_inputs(rng, (60,), d, n, 1, T[t])
    dy = randn(rng, 60, d, t=T[t])
    clean, want_clean = run_scan(v, lengths, dy), scan_values(v, lengths, dy)
    (dy if where == "dy" else v[where])[t0, c0] = value
    want = scan_values(v, lengths, dy)
    if where in ("x", "dy"):
        assert np.isfinite(want["dB" if where == "x" else "dC"]).all((1, 2)).sum() == 59  # one row of 60
    same_where_finite(run_scan(v, lengths, dy), clean, want, want_clean, "%s %s" % (where, value))


def positive(v):
    """Every term of one sign, so that an infinity stays one: no difference of infinities but the formulas' own."""
    return {k: (q if k == "A" or q is None else q.abs()) for k, q in v.items()}


def same_kind(got, want, what):
    """Infinite, not a number or finite exactly where the formulas are."""
    for name, q in got.items():
        w = torch.from_numpy(np.asarray(want[name])).view(q.shape)
        q = q.double().cpu()
        for kind in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(kind(q), kind(w)), "%s %s %s" % (what, name, kind.__name__)


@pytest.mark.parametrize("n", [1, 5, 13, 16, 24, 40, 64])
@pytest.mark.parametrize("where", ["x", "delta", "dy"])
def test_infinities_do_not_meet_the_padding_of_the_states(where, n):
    """An infinite input gives the same with 13 states as with 16: states are padded to 16, 32 or 64 with
    zeros, and zero times infinity is no zero."""
    rng = np.random.default_rng(70 + n)
    lengths, d, t0, c0 = [40, 20], 24, 21, 11
    v = positive(scan_inputs(rng, (60,), d, n))
    dy = randn(rng, 60, d).abs()
    (dy if where == "dy" else v[where])[t0, c0] = float("inf")
    same_kind(run_scan(v, lengths, dy), scan_values(v, lengths, dy), where)


@pytest.mark.parametrize("n", [1, 5, 16, 24, 40])
@pytest.mark.parametrize("rows", [3, 2051])
def test_step_infinities_do_not_meet_the_padding_of_the_states(rows, n):
    rng = np.random.default_rng(80 + n)
    d = 130
    v = positive(scan_inputs(rng, (rows,), d, n))
    v["x"][1, 7] = float("inf")
    state = torch.zeros(rows, d, n, device="cuda")
    a, kw = call_args(v)
    y = dw.selective_scan_step(*a, state, delta_softplus=True, **kw)
    want = scan_values(v, [1] * rows)
    same_kind(dict(y=y, final=state), want, "step")


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("with_z", [True, False])
def test_infinite_gradient_without_skip(n, with_z):
    """Without D dx has no term of it, as y has none: 0 times an infinite dy is not zero."""
    rng = np.random.default_rng(90 + n)
    lengths, d = [40, 20], 40
    v = positive(scan_inputs(rng, (60,), d, n))
    v["D"] = None
    if not with_z:
        v["z"] = None
    dy = randn(rng, 60, d).abs()
    dy[21, 5] = float("inf")
    got, want = run_scan(v, lengths, dy), scan_values(v, lengths, dy)
    assert np.isposinf(want["dx"][21, 5])
    same_kind(got, {k: want[k] for k in got}, "no D")


@pytest.mark.parametrize("n", [1, 16, 24, 64])
@pytest.mark.parametrize("where", ["x", "dfinal"])
def test_infinities_do_not_meet_the_rows_behind_a_sequence(where, n):
    """A sequence that ends inside four rows: the rows behind it take no part, so an infinite state at its
    last row does not reach dA, which has no term of that state."""
    rng = np.random.default_rng(100 + n)
    lengths, d = [22, 5, 35], 40
    v = positive(scan_inputs(rng, (62,), d, n))
    dy, dfin = randn(rng, 62, d).abs(), randn(rng, 3, d, n).abs()
    if where == "x":
        v["x"][21, 5] = v["x"][26, 30] = float("inf")
    else:
        dfin[0, 5], dfin[1, 30] = float("inf"), float("inf")
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=offsets(lengths))
    g = {k: q for k, q in dw.selective_scan_grad(dy, *a, dfinal_state=dfin, **kw)._asdict().items() if q is not None}
    want = scan_values(v, lengths, dy, dfinal=dfin)
    if where == "x":
        assert np.isfinite(want["dA"]).all()
    same_kind(g, {k: want[k] for k in g}, where)


@pytest.mark.parametrize("n", [3, 16, 40])
def test_rate_of_minus_infinity_forgets(n):
    """A = -inf gives the factor 0, as any rate does whose exponential underflows: also where a tile ends
    inside a sequence, whose remaining rows have a step of zero."""
    rng = np.random.default_rng(110 + n)
    lengths, d = [22, 5, 135], 40
    v = scan_inputs(rng, (162,), d, n)
    init = randn(rng, 3, d, n)
    got = []
    for rate in (-float("inf"), -1e30):
        v["A"][7, 0] = v["A"][33, n - 1] = rate
        a, kw = call_args(v)
        kw.update(delta_softplus=True, seq_offsets=offsets(lengths), initial_state=init)
        y, fin = dw.selective_scan(*a, final_state=True, **kw)
        state = init.clone()
        step = dw.selective_scan_step(*[q[:3] if q.shape[0] == 162 else q for q in a], state, D=v["D"], z=v["z"][:3],
                                      delta_bias=v["delta_bias"], delta_softplus=True)
        got.append((y, fin, step, state))
    for p, q in zip(*got):
        assert torch.isfinite(p).all() and torch.equal(p, q)


# ---------------------------------------------------------------------- more workgroups than one dimension of a grid holds
def test_lookup_of_more_tokens_than_a_grid_row():
    n = (1 << 26) + 5
    table = torch.arange(1, 12, dtype=torch.float16, device="cuda")[:, None]
    tok = (torch.arange(n, dtype=torch.int32, device="cuda") % 13) - 1  # -1 and 11 are outside the table
    y = dw.embedding_lookup(tok, table, scale=2.0)
    want = torch.where((tok >= 0) & (tok < 11), (tok + 1) * 2, 0).to(torch.float16)
    assert torch.equal(y[:, 0], want)


def test_table_gradient_of_more_rows_than_a_grid_row():
    v, d = 1 << 24, 1023  # odd: one element per lane
    tok = torch.tensor([0, v - 1, 12345678, v - 1, -1, v], dtype=torch.int32, device="cuda")
    dout = torch.randint(-8, 9, (6, d), device="cuda").to(torch.bfloat16)
    g = dw.embedding_grad(tok, dout, v)
    for r, want in ((0, dout[0]), (12345678, dout[2]), (v - 1, dout[1] + dout[3])):
        assert torch.equal(g[r], want)
        g[r] = 0
    assert not g.any()


def test_convolution_of_more_sequences_than_a_grid_row():
    b = (1 << 29) + 3
    x = (torch.arange(b, dtype=torch.int32, device="cuda") % 251).to(torch.bfloat16).view(b, 1, 1)
    w = torch.tensor([[3.0, 0.5]], dtype=torch.bfloat16, device="cuda")
    y, fin = dw.causal_conv1d(x, w, final_state=True)
    assert torch.equal(fin, x) and torch.equal(y, x * 0.5)


def test_scan_of_more_sequences_than_a_grid_row():
    b = (1 << 24) + 3
    one = torch.ones(b, 1, 1, device="cuda")
    x = (torch.arange(b, dtype=torch.int32, device="cuda") % 1021).float().view(b, 1, 1)
    args = (x, one, -torch.ones(1, 1, device="cuda"), one[..., None], one[..., None])
    y, fin, saved = dw.selective_scan(*args, final_state=True, save_for_grad=True)
    assert torch.equal(y, x) and torch.equal(fin, x)  # dt x B = x
    g = dw.selective_scan_grad(x, *args, saved=saved)
    assert torch.equal(g.dx, x) and torch.equal(g.dC[..., 0], x * x) and torch.equal(g.dB[..., 0], x * x)
    state = torch.zeros(b, 1, 1, device="cuda")
    step = dw.selective_scan_step(x[:, 0], one[:, 0], args[2], one, one, state)
    assert torch.equal(step, x[:, 0]) and torch.equal(state, x)


# ---------------------------------------------------------------------- autograd
def test_parameters_are_refused_where_autograd_records():
    rng = np.random.default_rng(120)
    x, w = randn(rng, 2, 6, 16), torch.nn.Parameter(randn(rng, 16, 4))
    table, tok = torch.nn.Parameter(randn(rng, 9, 16)), torch.zeros(3, dtype=torch.int32, device="cuda")
    A, bc = torch.nn.Parameter(-randn(rng, 16, 8).abs()), randn(rng, 2, 6, 1, 8)
    calls = [lambda: dw.embedding_lookup(tok, table), lambda: dw.causal_conv1d(x, w), lambda: dw.causal_conv1d_grad(x, x, w),
             lambda: dw.causal_conv1d_step(x[:, 0], x[:, :3].contiguous(), w), lambda: dw.selective_scan(x, x, A, bc, bc),
             lambda: dw.selective_scan_grad(x, x, x, A, bc, bc), lambda: dw.embedding_grad(tok, table[:3], 9),
             lambda: dw.selective_scan_step(x[:, 0], x[:, 0], A, bc[:, 0], bc[:, 0], torch.zeros(2, 16, 8, device="cuda"))]
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()

    class Conv(torch.autograd.Function):  # the way into a graph: both directions run outside of it
        @staticmethod
        def forward(ctx, x, w):
            ctx.save_for_backward(x, w)
            return dw.causal_conv1d(x, w, activation="silu")

        @staticmethod
        def backward(ctx, dy):
            g = dw.causal_conv1d_grad(dy.contiguous(), *ctx.saved_tensors, activation="silu")
            return g.dx, g.dweight
    dy = randn(rng, 2, 6, 16)
    Conv.apply(x, w).backward(dy)
    with torch.no_grad():
        assert torch.equal(w.grad, dw.causal_conv1d_grad(dy, x, w, activation="silu").dweight)


# ---------------------------------------------------------------------- rows of no sequence
@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_new_gradients_of_rows_without_a_sequence_are_zero(t):
    """Whatever the allocator hands out: no output depends on those rows."""
    rng = np.random.default_rng(130)
    rows, d, n, lo, hi, t = 120, 64, 16, 3, 100, T[t]
    v = scan_inputs(rng, (rows,), d, n, 2, t)
    dy, w = randn(rng, rows, d, t=t), randn(rng, d, 4, t=t)
    off = offsets([50, 0, 47], lo)
    a, kw = call_args(v)
    for _ in range(2):
        junk = [torch.full(s, float("nan"), dtype=t, device="cuda") for s in [(rows, d)] * 8 + [(rows, 2, n)] * 4]
        del junk
        g = dw.selective_scan_grad(dy, *a, delta_softplus=True, seq_offsets=off, **kw)
        c = dw.causal_conv1d_grad(dy, v["x"], w, seq_offsets=off)
        for q in (g.dx, g.ddelta, g.dz, g.dB, g.dC, c.dx):
            assert (q[:lo] == 0).all() and (q[hi:] == 0).all() and torch.isfinite(q).all() and q[lo:hi].any()


# ---------------------------------------------------------------------- precision
@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("lengths,d,n", [([300, 2, 211], 24, 16), ([33, 64, 5], 72, 16), ([1500], 40, 16), ([700, 90], 40, 5), ([512], 24, 40),
                                         ([129, 0, 400], 16, 64)])
def test_scan_errors_do_not_grow_with_the_length(t, lengths, d, n):
    """Within bounds that follow the recurrence (tests/test_sequence_errors_host.py shows that a state of
    16 bits leaves them): no state, sum or factor is held in fewer than 32."""
    rng = np.random.default_rng(sum(lengths) + n)
    rows, t = sum(lengths), T[t]
    v = scan_inputs(rng, (rows,), d, n, 1, t)
    init, dfin, dy = randn(rng, len(lengths), d, n), randn(rng, len(lengths), d, n), randn(rng, rows, d, t=t)
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=offsets(lengths), initial_state=init)
    y, fin, saved = dw.selective_scan(*a, final_state=True, save_for_grad=True, **kw)
    g = dw.selective_scan_grad(dy, *a, saved=saved, dfinal_state=dfin, **kw)._asdict()
    g["dinitial"] = g.pop("dinitial_state")
    ends = np.cumsum([0] + lengths)
    want = err.scan(f64(v["x"]), f64(v["delta"]), f64(v["A"]), f64(v["B"]), f64(v["C"]), f64(v["D"]), f64(v["z"]), f64(v["delta_bias"]), True,
                    list(zip(ends[:-1], ends[1:])), f64(init), f64(dy), f64(dfin))
    for name, q in dict(g, y=y, final=fin).items():
        err.near(q, *want[name], name)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_convolution_parameter_sums_of_long_blocks(t):
    """Enough rows for the longest row blocks: dweight and dbias within the bounds of their own terms, which
    a block left out leaves."""
    rng = np.random.default_rng(131)
    b, l, d, some, t = 64, 700, 1024, slice(480, 544), T[t]
    x, dy = randn(rng, b, l, d, t=t), randn(rng, b, l, d, t=t)
    w, bias = randn(rng, d, 4, t=t), randn(rng, d, t=t)
    g = dw.causal_conv1d_grad(dy, x, w, bias, activation="silu")
    dweight, dbias, dweight_e, dbias_e = err.conv_sums(f64(x[..., some]), f64(dy[..., some]), f64(w[some]), f64(bias[some]))
    err.near(g.dweight[some], dweight, dweight_e, "dweight")
    err.near(g.dbias[some], dbias, dbias_e, "dbias")


# ---------------------------------------------------------------------- the vector path and the other one
@pytest.mark.parametrize("t", list(T))
def test_both_paths_give_the_same_bits_but_for_the_convolutions_sums(t):
    """The same values at whole 16-byte pieces and two bytes beside them, as the header says."""
    rng = np.random.default_rng(140)
    b, l, d, n, t = 3, 290, 64, 16, T[t]
    v = scan_inputs(rng, (b, l), d, n, 2, t)
    dy, w, bias = randn(rng, b, l, d, t=t), randn(rng, d, 4, t=t), randn(rng, d, t=t)

    def beside(q):
        wide = torch.zeros(q.shape[:2] + (q[0, 0].numel() + 1,), dtype=q.dtype, device="cuda")
        wide[..., 1:] = q.flatten(2)
        return wide[..., 1:].unflatten(-1, q.shape[2:]) if q.dim() == 4 else wide[..., 1:]
    a, kw = call_args(v)
    a2 = [beside(q) if q.dim() > 2 else q for q in a]
    kw2 = dict(kw, z=beside(v["z"]))
    for p, q in zip(dw.selective_scan(*a, delta_softplus=True, final_state=True, **kw),
                    dw.selective_scan(*a2, delta_softplus=True, final_state=True, **kw2)):
        assert torch.equal(p, q)
    for p, q in zip(dw.selective_scan_grad(dy, *a, delta_softplus=True, **kw),
                    dw.selective_scan_grad(beside(dy), *a2, delta_softplus=True, **kw2)):
        assert (p is None and q is None) or torch.equal(p, q)
    assert torch.equal(dw.causal_conv1d(v["x"], w, bias, activation="silu"), dw.causal_conv1d(a2[0], w, bias, activation="silu"))
    g, g2 = (dw.causal_conv1d_grad(r, x, w, bias, activation="silu") for r, x in ((dy, v["x"]), (beside(dy), a2[0])))
    assert torch.equal(g.dx, g2.dx)
    dweight, dbias, dweight_e, dbias_e = err.conv_sums(f64(v["x"]), f64(dy), f64(w), f64(bias))
    for q in (g, g2):
        err.near(q.dweight, dweight, dweight_e, "dweight")
        err.near(q.dbias, dbias, dbias_e, "dbias")


@pytest.mark.parametrize("packed", [True, False])
def test_no_sequences(packed):
    """Rows of no sequence, or a batch of none: nothing is written, sums over rows are zero."""
    rng = np.random.default_rng(150)
    d, n = 40, 16
    lead = (70,) if packed else (0, 7)
    v = scan_inputs(rng, lead, d, n)
    dy, w, bias = randn(rng, *lead, d), randn(rng, d, 4), randn(rng, d)
    off = torch.tensor([30], dtype=torch.int32, device="cuda") if packed else None
    a, kw = call_args(v)
    kw.update(delta_softplus=True, seq_offsets=off)
    out = torch.full(lead + (d,), 4.0, device="cuda")
    y, fin, saved = dw.selective_scan(*a, final_state=True, save_for_grad=True, out=out, **kw)
    assert (out == 4.0).all() and fin.shape == (0, d, n)
    g = dw.selective_scan_grad(dy, *a, saved=saved, **kw)
    y, cs = dw.causal_conv1d(v["x"], w, bias, seq_offsets=off, final_state=True, out=out)
    assert (out == 4.0).all() and cs.shape == (0, 3, d)
    c = dw.causal_conv1d_grad(dy, v["x"], w, bias, seq_offsets=off)
    for q in list(g) + list(c):
        assert q is None or not q.any()


@pytest.mark.parametrize("where", ["B", "C"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("d,n", [(48, 16), (40, 16), (20, 5), (24, 40)])
def test_scan_gradients_keep_a_state_to_itself(where, value, d, n):
    """A value of B or C that is not finite reaches its own state alone: of dA and dC (or dB), one column."""
    rng = np.random.default_rng(160 + n)
    lengths, t0, n0 = [41, 22], 21, n // 2
    v = scan_inputs(rng, (63,), d, n)
    dy = randn(rng, 63, d)
    clean, want_clean = run_scan(v, lengths, dy), scan_values(v, lengths, dy)
    v[where][t0, 0, n0] = value
    want = scan_values(v, lengths, dy)
    assert np.isfinite(want["dA"]).all(0).sum() == n - 1
    same_where_finite(run_scan(v, lengths, dy), clean, want, want_clean, "%s %s" % (where, value))


@pytest.mark.parametrize("where", ["x", "delta", "z", "dy"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_in_a_long_sequence(where, value):
    """The same across the spans that a long sequence is cut into."""
    rng = np.random.default_rng(170)
    lengths, d, n, t0, c0 = [403, 100], 24, 16, 210, 17
    v = scan_inputs(rng, (503,), d, n)
    dy = randn(rng, 503, d)
    clean, want_clean = run_scan(v, lengths, dy), scan_values(v, lengths, dy)
    (dy if where == "dy" else v[where])[t0, c0] = value
    got, want = run_scan(v, lengths, dy), scan_values(v, lengths, dy)
    same_where_finite(got, clean, want, want_clean, "%s %s" % (where, value))
