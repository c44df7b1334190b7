"""The error bounds of sequence_errors.py on the host: the formulas in 32 bits stay inside them, the same
formulas with a state of 16 bits, or with a block of rows left out of a sum, do not."""
import numpy as np
import pytest
import torch

import sequence_errors as err
import sequence_reference as ref


def inputs(rng, rows, d, n):
    f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    return dict(x=f(rows, d), delta=f(rows, d), A=-rng.uniform(0.2, 3.0, (d, n)).astype(np.float32), B=f(rows, 1, n), C=f(rows, 1, n),
                D=f(d), z=f(rows, d), bias=f(d) - np.float32(2.0))


def in_32_bits(v, seqs, dy, state=torch.float32, adjoint=torch.float32):
    """y and dx by rows in 32 bits, the state and its gradient rounded to these types after every row."""
    t = {k: torch.from_numpy(q) for k, q in v.items()}
    dt = torch.nn.functional.softplus(t["delta"] + t["bias"])
    a = torch.exp(dt[..., None] * t["A"])
    gate = torch.nn.functional.silu(t["z"])
    y, dx = torch.zeros_like(t["x"]), torch.zeros_like(t["x"])
    for lo, hi in seqs:
        h = torch.zeros_like(t["A"])
        for r in range(lo, hi):
            h = (a[r] * h + (dt[r] * t["x"][r])[:, None] * t["B"][r]).to(state).float()
            y[r] = ((h * t["C"][r]).sum(-1) + t["D"] * t["x"][r]) * gate[r]
        g = torch.zeros_like(t["A"])
        for r in range(hi - 1, lo - 1, -1):
            dv = dy[r] * gate[r]
            dh = (dv[:, None] * t["C"][r] + g).to(adjoint).float()
            dx[r] = dv * t["D"] + dt[r] * (dh * t["B"][r]).sum(-1)
            g = a[r] * dh
    return {"y": y.double().numpy(), "dx": dx.double().numpy()}


@pytest.mark.parametrize("lengths", [[300, 2, 211], [33, 64, 5], [1500]])
def test_bounds_hold_in_32_bits_and_show_a_16_bit_state(lengths):
    rng = np.random.default_rng(sum(lengths))
    rows, d, n = sum(lengths), 24, 16
    ends = np.cumsum([0] + lengths)
    seqs = list(zip(ends[:-1], ends[1:]))
    v = inputs(rng, rows, d, n)
    dy = rng.standard_normal((rows, d)).astype(np.float32)
    want = err.scan(**{k: ref.f64(torch.from_numpy(q)) for k, q in v.items()}, sp=True, seqs=seqs, dy=dy.astype(np.float64))
    right = in_32_bits(v, seqs, torch.from_numpy(dy))
    for name in ("y", "dx"):
        assert not err.outside(right[name], *want[name]).any(), name
    for name, kw in (("y", dict(state=torch.float16)), ("y", dict(state=torch.bfloat16)), ("dx", dict(adjoint=torch.float16))):
        wrong = in_32_bits(v, seqs, torch.from_numpy(dy), **kw)
        assert err.outside(wrong[name], *want[name]).mean() > 0.3, (name, kw)


def test_bounds_of_the_parameter_sums_show_a_block_left_out():
    rng = np.random.default_rng(3)
    b, l, d, k = 64, 700, 8, 4
    x, dy = rng.standard_normal((b, l, d)), rng.standard_normal((b, l, d))
    w, bias = rng.standard_normal((d, k)), rng.standard_normal(d)
    dw, db, dw_e, db_e = err.conv_sums(x, dy, w, bias)
    # against autograd
    t = [torch.from_numpy(q).requires_grad_(i > 0) for i, q in enumerate((x, w, bias))]
    u = t[2] + (torch.nn.functional.pad(t[0], (0, 0, k - 1, 0)).unfold(1, k, 1) * t[1]).sum(-1)
    gw, gb = torch.autograd.grad(torch.nn.functional.silu(u), t[1:], torch.from_numpy(dy))
    np.testing.assert_allclose(gw.numpy(), dw, rtol=1e-10, atol=1e-9)
    np.testing.assert_allclose(gb.numpy(), db, rtol=1e-10, atol=1e-9)
    for first in (0, 128 * 100, 128 * 349):
        less_w, less_b = err.conv_sums(x, dy, w, bias, slice(first, first + 128))[:2]
        assert (np.abs(less_w - dw) > dw_e).mean() > 0.8 and (np.abs(less_b - db) > db_e).mean() > 0.5
