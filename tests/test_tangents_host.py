"""Tensors with a tangent (forward-mode differentiation) are refused by every sequence operator before anything runs, like
those that require a gradient; others are not, inside a level too."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import device_wide_prefix_tile_amd as dw
from device_wide_prefix_tile_amd import sequence as seq


def cases():
    x, row = torch.zeros(2, 3, 8), torch.zeros(3, 8)
    rate, ints = torch.zeros(8), torch.zeros(3, 2, dtype=torch.int32)
    plan = dw.ExpertPlan(torch.zeros(5, dtype=torch.int32), ints, ints.view(-1))
    A, B = torch.zeros(8, 4), torch.zeros(2, 3, 1, 4)
    return [("embedding_lookup", (ints, row), 1), ("causal_conv1d", (x, torch.zeros(8, 4)), 0), ("selective_scan", (x, x, A, B, B), 0),
            ("gated_scan", (x, x, x, rate), 0), ("gated_scan_step", (row, row, row, rate, row), 0), ("expert_dispatch", (row, plan), 0),
            ("expert_combine", (row, plan), 0), ("expert_dispatch_grad", (row, plan), 0), ("expert_combine_grad", (row, row, plan), 0),
            ("sample_tokens", (row, row[:, 0]), 0)]


@pytest.mark.parametrize("name,args,at", cases(), ids=lambda v: v if isinstance(v, str) else "")
def test_tangents_are_refused(name, args, at):
    f = getattr(dw, name)
    with pytest.raises((ValueError, TypeError)) as plain:
        f(*args)
    assert "tangent" not in str(plain.value)  # for its device
    with fwad.dual_level():
        with pytest.raises((ValueError, TypeError)) as inside:
            f(*args)
        assert "tangent" not in str(inside.value)
        dual = list(args)
        dual[at] = fwad.make_dual(args[at].clone(), torch.ones_like(args[at]))
        for mode in (torch.enable_grad, torch.no_grad):
            if name == "embedding_lookup":
                with mode(), pytest.raises(ValueError, match="table has a tangent"):
                    seq._x(dual[at], "table")
            else:
                with mode(), pytest.raises(ValueError, match="has a tangent"):
                    f(*dual)


def test_every_kind_of_argument():
    """The checks that every other tensor of a call goes through: parameters, states, rows, outputs."""
    t = torch.zeros(4, 8)
    assert seq._plain(t, "t", (4, 8), torch.float32, -1) == t.data_ptr() and seq._like(t, "t", (4, 8), torch.float32, -1, 8)[0] == t.data_ptr()
    with fwad.dual_level():
        d = fwad.make_dual(t, torch.ones(4, 8))
        for check in (lambda q: seq._plain(q, "t", (4, 8), torch.float32, -1), lambda q: seq._like(q, "t", (4, 8), torch.float32, -1, 8)):
            check(t)
            with pytest.raises(ValueError, match="t has a tangent"):
                check(d)
            check(fwad.unpack_dual(d).primal)
