"""The gated recurrence without a GPU: the argument structures, the C ABI's refusals and sizes, and the 64-bit
reference: its gradients against differences, its bounds against the formulas in 32 bits."""
import ctypes

import numpy as np
import pytest
import torch

import gated_reference as gr
from device_wide_prefix_tile_amd import sequence as seq
from structure_check import check_structure

OK, INVALID, UNSUPPORTED = 0, 1, 2
MB = 1 << 20  # fake device addresses, a mebibyte apart: rejected calls never touch them


@pytest.fixture(scope="module")
def L():
    return seq._lib()


@pytest.mark.parametrize("name,cls", [("gated_scan_args_t", seq._GatedArgs), ("gated_scan_grad_args_t", seq._GatedGradArgs),
                                      ("gated_scan_step_args_t", seq._GatedStepArgs)])
def test_structures_match_the_header(name, cls):
    check_structure(name, cls, {"gated_scan_args_t": seq._GatedArgs})


def args(**kw):
    a = dict(dtype=2, rows=32, seqs=2, channels=64, x=MB, x_stride=64, decay_gate=2 * MB, decay_stride=64, input_gate=3 * MB, input_stride=64,
             rate=4 * MB, initial_state=5 * MB, y=6 * MB, y_stride=64, final_state=7 * MB, saved=8 * MB, workspace=9 * MB, workspace_bytes=MB)
    a.update(kw)
    return seq._GatedArgs(**a)


BAD = [dict(x=None), dict(decay_gate=None), dict(input_gate=None), dict(rate=None), dict(x=MB + 1), dict(decay_stride=63), dict(rate=4 * MB + 2),
       dict(channels=0), dict(channels=(1 << 20) + 1), dict(rows=33), dict(seqs=0), dict(rows=1 << 31), dict(seq_offsets=MB + 1),
       dict(initial_state=5 * MB + 1), dict(saved=8 * MB + 2), dict(x_stride=(1 << 31) + 1)]


def test_scan_refusals(L):
    call = lambda **kw: L.gated_scan(ctypes.byref(args(**kw)), None)  # noqa: E731
    assert L.gated_scan(None, None) == INVALID
    for bad in BAD + [dict(y=6 * MB + 1), dict(y_stride=1), dict(y=MB), dict(y=MB + 64), dict(final_state=5 * MB), dict(final_state=6 * MB),
                      dict(workspace=None), dict(workspace_bytes=255), dict(workspace=9 * MB + 8), dict(saved=6 * MB), dict(workspace=MB)]:
        assert call(**bad) == INVALID, bad
    assert call(dtype=3) == UNSUPPORTED and call(dtype=-1) == UNSUPPORTED


def test_grad_refusals(L):
    def call(fwd=(), **kw):
        g = dict(args=args(**dict(fwd)), dy=20 * MB, dy_stride=64, dfinal_state=21 * MB, dx=22 * MB, dx_stride=64, ddecay_gate=23 * MB,
                 ddecay_stride=64, dinput_gate=24 * MB, dinput_stride=64, drate=25 * MB, dinitial_state=26 * MB)
        g.update(kw)
        return L.gated_scan_grad(ctypes.byref(seq._GatedGradArgs(**g)), None)
    assert L.gated_scan_grad(None, None) == INVALID
    for bad in BAD + [dict(saved=None), dict(workspace=None), dict(workspace_bytes=256)]:
        assert call(fwd=bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dx=None), dict(ddecay_gate=None), dict(dinput_gate=None), dict(drate=None), dict(dx=20 * MB), dict(dx=MB),
                dict(dinput_gate=23 * MB), dict(ddecay_stride=3), dict(dinitial_state=21 * MB), dict(drate=25 * MB + 1), dict(dx=8 * MB)):
        assert call(**bad) == INVALID, bad


def test_step_refusals(L):
    def call(**kw):
        a = dict(dtype=0, rows=4, n_slots=9, slots=MB, channels=64, x=2 * MB, x_stride=64, decay_gate=3 * MB, decay_stride=64,
                 input_gate=4 * MB, input_stride=64, rate=5 * MB, state=6 * MB, y=7 * MB, y_stride=64)
        a.update(kw)
        return L.gated_scan_step(ctypes.byref(seq._GatedStepArgs(**a)), None)
    assert call(rows=0, x=None) == OK and L.gated_scan_step(None, None) == INVALID
    for bad in (dict(x=None), dict(decay_gate=None), dict(rate=None), dict(state=None), dict(y=None), dict(y=2 * MB), dict(state=7 * MB),
                dict(y_stride=1), dict(state=6 * MB + 2), dict(n_slots=1 << 31), dict(slots=MB + 2), dict(rows=1 << 31), dict(channels=0)):
        assert call(**bad) == INVALID, bad
    assert call(dtype=9) == UNSUPPORTED


def test_sizes(L):
    """One tile of rows waits for nothing; more of them hold a map per channel and tile."""
    ws = lambda **kw: L.gated_scan_workspace(ctypes.byref(args(**kw)))  # noqa: E731
    assert ws() == 256 and ws(rows=128) == 256
    assert ws(rows=130) >= 4 * 256 * 8  # two sequences of 65 rows: two tiles each
    assert ws(rows=33) == 0
    assert L.gated_scan_saved(ctypes.byref(args(rows=130))) == 4 * 8 * 256
    assert L.gated_scan_saved(ctypes.byref(args(rows=0, seqs=0, x=None, decay_gate=None, input_gate=None))) == 0
    assert L.gated_scan_grad_workspace(ctypes.byref(args(rows=130))) >= ws(rows=130) + 4 * 256 * 4
    # no sequences is a call where offsets say so
    assert L.gated_scan_workspace(ctypes.byref(args(seqs=0, seq_offsets=16 * MB))) > 0


def test_tensors_that_require_gradients_are_refused():
    x = torch.zeros(1, 4, 8, requires_grad=True)
    import device_wide_prefix_tile_amd as dw
    with pytest.raises(ValueError, match="requires a gradient"):
        dw.gated_scan(x, x, x, torch.zeros(8))
    with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):
        dw.gated_scan(x, x, x, torch.zeros(8))


def sample(rng, rows, d):
    return dict(x=rng.standard_normal((rows, d)), decay=2 * rng.standard_normal((rows, d)), inp=rng.standard_normal((rows, d)),
                rate=-np.exp(rng.uniform(np.log(1e-2), np.log(4.0), d)))


def test_reference_gradients_match_differences():
    rng = np.random.default_rng(3)
    rows, d = 11, 6
    seqs = [(0, 4), (4, 4), (4, 5), (5, 11)]
    v = dict(sample(rng, rows, d), initial=rng.standard_normal((4, d)))
    dy, dfin = rng.standard_normal((rows, d)), rng.standard_normal((4, d))

    def loss(**kw):
        r = gr.gated(seqs=seqs, **kw)
        return (r["y"][0] * dy).sum() + (r["final"][0] * dfin).sum()
    grads = gr.gated(seqs=seqs, dy=dy, dfinal=dfin, **v)
    for name, of in (("x", "dx"), ("decay", "ddecay"), ("inp", "dinput"), ("rate", "drate"), ("initial", "dinitial")):
        h, step = 1e-6, rng.standard_normal(v[name].shape)
        up, down = dict(v), dict(v)
        up[name], down[name] = v[name] + h * step, v[name] - h * step
        got = (loss(**up) - loss(**down)) / (2 * h)
        # central differences: h^2 of the third derivative, and 2^-52 / h of the loss's terms
        assert abs(got - (grads[of][0] * step).sum()) <= 1e-7 * (1 + np.abs(grads[of][0] * step).sum()), name


def test_bounds_hold_in_32_bits_and_show_a_16_bit_state():
    rng = np.random.default_rng(4)
    rows, d = 900, 32
    v = {k: q.astype(np.float32) for k, q in sample(rng, rows, d).items()}
    dy = rng.standard_normal((rows, d)).astype(np.float32)
    want = gr.gated(**{k: q.astype(np.float64) for k, q in v.items()}, seqs=[(0, rows)], dy=dy.astype(np.float64))
    t = {k: torch.from_numpy(q) for k, q in v.items()}
    f, g = torch.sigmoid(t["decay"]), torch.sigmoid(t["inp"])
    a, w = torch.exp(t["rate"] * f), torch.sqrt(-torch.expm1(2 * t["rate"] * f))
    for held, right in ((torch.float32, True), (torch.float16, False), (torch.bfloat16, False)):
        h, e = torch.zeros(d), torch.zeros(d)
        y, dx = torch.zeros(rows, d), torch.zeros(rows, d)
        for r in range(rows):
            h = (a[r] * h + w[r] * g[r] * t["x"][r]).to(held).float()
            y[r] = h
        for r in range(rows - 1, -1, -1):
            dh = (torch.from_numpy(dy[r]) + e).to(held).float()
            dx[r] = dh * w[r] * g[r]
            e = a[r] * dh
        for got, name in ((y, "y"), (dx, "dx")):
            val, err = want[name]
            out = np.abs(got.double().numpy() - val) > err + gr.U * np.abs(val)
            assert not out.any() if right else out.mean() > 0.3, (name, held)
