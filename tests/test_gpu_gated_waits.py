"""Waits of the gated recurrence that give up: every kernel still ends, the results say so, and so does the device's word."""
import pytest
import torch

import device_wide_prefix_tile_amd as dw

pytestmark = pytest.mark.gpu

OK, TIMEOUT = 0, 5


def test_waits_that_give_up_are_reported():
    gen = torch.Generator(device="cuda").manual_seed(3)
    rows, d = 700, 200  # eleven tiles of 64 rows: a group of eight and one of three
    x, u, v, dy = (torch.randn(1, rows, d, generator=gen, device="cuda") for _ in range(4))
    args = (x, u, v, -torch.rand(d, generator=gen, device="cuda"))
    want, saved = dw.gated_scan(*args, save_for_grad=True)
    grads = dw.gated_scan_grad(dy, *args, saved=saved)
    assert dw.seq_get_device_error() == OK
    old = dw.seq_set_spin_limit(0)
    try:
        y = dw.gated_scan(*args)
        assert dw.seq_get_device_error() == TIMEOUT and dw.seq_get_device_error() == OK
        assert torch.equal(y[:, :64], want[:, :64]) and y[:, 64:].isnan().all()
        g = dw.gated_scan_grad(dy, *args, saved=saved)
        assert dw.seq_get_device_error(torch.cuda.current_stream()) == TIMEOUT and dw.seq_get_device_error() == OK
        assert torch.equal(g.dx[:, 640:], grads.dx[:, 640:]) and g.dx[:, :640].isnan().all()
        # nothing to wait for: single tiles, and runs that a workgroup walks through whole
        dw.gated_scan(*[q[:, :64] for q in args[:3]], args[3])
        many = [q[:, :65, :64].expand(300, -1, -1).contiguous() for q in (dy, x, u, v)]
        r = -torch.ones(64, device="cuda")
        states = torch.zeros(300 * 2 * 8 * 256, device="cuda")
        dw.gated_scan_grad(*many, r, saved=states)
        assert dw.seq_get_device_error() == OK
    finally:
        assert dw.seq_set_spin_limit(old) == 0
    again, saved = dw.gated_scan(*args, save_for_grad=True)
    assert torch.equal(again, want) and all(p is None or torch.equal(p, q) for p, q in zip(dw.gated_scan_grad(dy, *args, saved=saved), grads))
    assert dw.seq_get_device_error() == OK and dw.seq_set_spin_limit(old) == old == 1 << 22
