"""The gated recurrence at gates so nearly closed that 1 - a^2 is below the smallest normal number, against the formulas in
64 bits (gated_reference.py)."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import gated_reference as gr
from gated_batch import T, named, randn, reference
from sequence_errors import near
from sequence_reference import f64

pytestmark = pytest.mark.gpu


def more(v, dy):
    """What the reference does not know of, per result: the relative error `low` of w = sqrt(1 - a^2) and of 1 / w next to
    a closed gate, in the terms that hold them: w g x, and a g x f / w times dh.

    1 - a^2 = 2 |rate| f there.  Below 2^-126 every product is rounded to a multiple of 2^-149, an error of 2^-150: of rate
    log2 e, of y = that times f, of a y (each relative to y = (1 - a^2) / (2 ln 2)) and of that times the series, together
    (3 2 ln 2 + 1) 2^-150 / (1 - a^2), and half of it in the root: 2.6 2^-150 / (1 - a^2), of which 4 are taken.
    Where f is below 2^-125 it may be flushed to 0 and w with it: all of w, of which the reference counts 0.9 (half of
    1.5, as for a small error)."""
    f, g = gr.sigmoid(f64(v[1])), gr.sigmoid(f64(v[2]))
    rate = f64(v[3])
    z = rate * f
    a, w, gx = np.exp(z), np.sqrt(-np.expm1(2 * z)), np.abs(g * f64(v[0]))
    low = np.where(f < 2.0 ** -125, 1.0, np.minimum(1.0, 4 * 2.0 ** -150 / np.maximum(2 * np.abs(z), 1e-300)))
    dh, h = np.zeros_like(f), np.zeros_like(f)
    e = np.zeros_like(f[:, 0])
    for r in range(f.shape[1] - 1, -1, -1):
        dh[:, r] = np.abs(f64(dy)[:, r]) + e
        e = a[:, r] * dh[:, r]
    e = np.zeros_like(e)
    for r in range(f.shape[1]):
        e = h[:, r] = a[:, r] * e + (w * gx * low)[:, r]
    slope = dh * gx * f / w * low + dh * f * (h / a)  # the state's own error
    return low, dict(y=h, dx=dh * w * g * low, dinput=dh * w * gx * low, ddecay=slope * np.abs(rate), drate=slope.sum((0, 1)), dinitial=0.0)


def check_more(got, want, extra, what):
    for name, q in got.items():
        assert torch.isfinite(q).all(), "%s %s" % (what, name)
        near(q, want[name][0], want[name][1] + extra[name], "%s %s" % (what, name))


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l", [(1, 200), (4, 50), (300, 66)], ids=["long", "batch", "runs"])
def test_nearly_closed_gates(t, b, l):
    """Decay gates from -90 to -70 in steps of a quarter, beside rows with open ones, at rates of every size."""
    rng = np.random.default_rng(b)
    d, t = 12, T[t]
    v = [randn(rng, b, l, d, t=t) for _ in range(3)]
    steps = torch.arange(-90, -69.9, 0.25, device="cuda").to(t)
    at = torch.from_numpy(rng.integers(0, steps.numel(), (b, l, d))).cuda()
    closed = torch.from_numpy(rng.random((b, l, d)) < 0.5).cuda()
    v[1] = torch.where(closed, steps[at], v[1])
    v[1][:, :3] = steps[at][:, :3]  # nothing but a closed gate's input in the state
    v.append(torch.tensor([-0.008, -0.1, -0.8, -1e-3, -8.0, -0.01] * 2, device="cuda"))
    dy, init = randn(rng, b, l, d, t=t), randn(rng, b, d)
    for start in (init, None):
        y, saved = dw.gated_scan(*v, initial_state=start, save_for_grad=True)
        g = dw.gated_scan_grad(dy, *v, initial_state=start, saved=saved)
        check_more(dict(named(g), y=y), reference(v, start, dy), more(v, dy)[1], "closed gates")


def test_rates_next_to_zero():
    """A rate whose 1 - a^2 is below the normal numbers at an open gate: the root's derivative is large, not infinite."""
    rng = np.random.default_rng(7)
    b, l, d = 2, 70, 6
    v = [randn(rng, b, l, d) for _ in range(3)] + [torch.tensor([-1e-38, -3e-39, -1e-40, -1e-36, -1e-30, -1e-12], device="cuda")]
    dy = randn(rng, b, l, d)
    low, extra = more(v, dy)
    assert 1e-6 < low.max() < 1e-3
    y, saved = dw.gated_scan(*v, save_for_grad=True)
    check_more(dict(named(dw.gated_scan_grad(dy, *v, saved=saved)), y=y), reference(v, None, dy), extra, "rates next to zero")
