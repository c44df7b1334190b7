"""The gated recurrence's gradient on long runs that workgroups walk through whole, against the formulas in 64 bits
(gated_reference.py)."""
import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
from gated_batch import T, check, named, randn, reference

pytestmark = pytest.mark.gpu


def test_rates_sums_over_long_runs():
    """Equal terms, whose plain sum in 32 bits is off by an amount that grows with their number (some 450 units of 2^-24
    after 4096 of them): the sum's own error stays at the few roundings that the reference counts."""
    l, d, t = 32768, 16384, torch.bfloat16
    x = torch.empty(1, l, d, dtype=t, device="cuda")
    rng = np.random.default_rng(11)
    values = [torch.from_numpy(rng.uniform(0.5, 1.0, d)).to(t).cuda() for _ in range(4)]
    v = [x.copy_(values[0]), x.clone().copy_(values[1]), x.clone().copy_(values[2]),
         -torch.from_numpy(rng.uniform(0.05, 0.5, d)).float().cuda()]
    dy = x.clone().copy_(values[3])
    y, saved = dw.gated_scan(*v, save_for_grad=True)
    g = dw.gated_scan_grad(dy, *v, saved=saved)
    some = torch.arange(0, d, d // 16, device="cuda")
    pick = lambda q: q[..., some]  # noqa: E731
    want = reference([pick(q) for q in v], None, pick(dy))
    check({k: pick(q) for k, q in dict(named(g), y=y).items()}, want, "long runs")


@pytest.mark.parametrize("t", list(T))
@pytest.mark.parametrize("b,l,d", [(8, 2049, 4096), (256, 3000, 64), (100, 1500, 200)])
def test_whole_runs_of_thousands_of_rows(t, b, l, d):
    """Dozens of tiles one after another, the last one of few rows; one and two channels per lane."""
    rng = np.random.default_rng(b + d)
    gen = torch.Generator(device="cuda").manual_seed(b + d)
    t = T[t]
    v = [(torch.randn(b, l, d, generator=gen, device="cuda") * s).to(t) for s in (1.0, 2.0, 2.0)]
    v.append(-torch.from_numpy(np.exp(rng.uniform(np.log(1e-3), np.log(4.0), d))).float().cuda())
    dy = torch.randn(b, l, d, generator=gen, device="cuda").to(t)
    init, dfin = randn(rng, b, d), randn(rng, b, d)
    y, fin, saved = dw.gated_scan(*v, initial_state=init, final_state=True, save_for_grad=True)
    g = dw.gated_scan_grad(dy, *v, initial_state=init, dfinal_state=dfin, saved=saved)
    some = torch.tensor([0, d // 2 - 1, d - 1], device="cuda")
    pick = lambda q: q[..., some].contiguous()  # noqa: E731
    want = reference([pick(q) for q in v], pick(init), pick(dy), pick(dfin))
    check({k: pick(q) for k, q in dict(named(g), y=y, final=fin).items()}, want, "whole runs")
    for _ in range(3):
        again = dw.gated_scan_grad(dy, *v, initial_state=init, dfinal_state=dfin, saved=saved)
        for p, q in zip(g, again):
            assert torch.equal(p, q)
