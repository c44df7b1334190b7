"""Batches of the gated recurrence against gated_reference.py, sequences of one length side by side."""
import numpy as np
import torch

import gated_reference as gr
from sequence_errors import near
from sequence_reference import f64

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(rng, *shape, t=torch.float32, scale=1.0):
    return (torch.from_numpy(rng.standard_normal(shape)) * scale).to(t).cuda()


def folded(q):
    """(B, L, D) as one sequence of L rows with B D channels."""
    return f64(q).transpose(1, 0, 2).reshape(q.shape[1], -1)


def reference(v, init=None, dy=None, dfinal=None):
    """The reference of a batch: its sequences side by side as channels; rates' gradients and their errors added up."""
    b, l, d = v[0].shape
    flat = lambda q: None if q is None else f64(q).reshape(1, -1)  # noqa: E731
    r = gr.gated(*[folded(q) for q in v[:3]], np.tile(f64(v[3]), b), [(0, l)], flat(init), None if dy is None else folded(dy), flat(dfinal))
    out = {}
    for name, pair in r.items():
        if name == "drate":
            out[name] = tuple(q.reshape(b, d).sum(0) for q in pair)
        elif name in ("final", "dinitial"):
            out[name] = tuple(q.reshape(b, d) for q in pair)
        else:
            out[name] = tuple(q.reshape(l, b, d).transpose(1, 0, 2) for q in pair)
    return out


def named(g):
    r = dict(dx=g.dx, ddecay=g.ddecay_gate, dinput=g.dinput_gate, drate=g.drate)
    if g.dinitial_state is not None:
        r["dinitial"] = g.dinitial_state
    return r


def check(got, want, what):
    for name, g in got.items():
        near(g, *want[name], "%s %s" % (what, name))
