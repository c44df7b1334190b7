"""Experts and sampling without a GPU: the argument structures, refusals of the C ABI and of the binding, sizes, and the
64-bit reference of sampling on rows worked out by hand."""
import ctypes

import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sampling_reference as sr
from device_wide_prefix_tile_amd import experts, sampling, sequence as seq
from structure_check import check_structure

OK, INVALID, UNSUPPORTED = 0, 1, 2
MB = 1 << 20  # fake device addresses, a mebibyte apart: rejected calls never touch them


@pytest.fixture(scope="module")
def L():
    return seq._lib()


@pytest.mark.parametrize("name,cls", [("expert_dispatch_args_t", experts._DispatchArgs), ("expert_combine_args_t", experts._CombineArgs),
                                      ("expert_combine_grad_args_t", experts._CombineGradArgs), ("sample_tokens_args_t", sampling._SampleArgs)])
def test_structures_match_the_header(name, cls):
    check_structure(name, cls)


def test_split_refusals(L):
    need = L.expert_split_workspace(5000, 64)

    def call(e=MB, n=5000, k=64, offsets=2 * MB, places=3 * MB, source=4 * MB, ws=5 * MB, wb=need):
        return L.expert_split(e, n, k, offsets, places, source, ws, wb, None)
    for bad in (dict(e=None), dict(e=MB + 2), dict(n=1 << 31), dict(k=0), dict(k=1025), dict(offsets=None), dict(places=None), dict(source=None),
                dict(offsets=2 * MB + 1), dict(places=MB), dict(source=3 * MB + 400), dict(offsets=4 * MB), dict(ws=None), dict(ws=5 * MB + 4),
                dict(wb=need - 1), dict(ws=3 * MB)):
        assert call(**bad) == INVALID, bad
    # one chunk of choices needs no counts
    assert L.expert_split_workspace(4096, 1024) == 0 < need
    assert L.expert_split_workspace(4097, 64) >= 2 * 64 * 4
    assert call(k=1025, wb=1 << 40) == INVALID == call(n=1 << 31, wb=1 << 60)


MOVES_BAD = [dict(choices=0), dict(choices=257), dict(channels=0), dict(channels=(1 << 20) + 1), dict(places=None), dict(places=MB + 1),
             dict(tokens=1 << 30), dict(rows=1 << 31)]


def test_dispatch_refusals(L):
    def call(**kw):
        a = dict(dtype=2, tokens=16, rows=32, choices=2, channels=64, places=MB, used=2 * MB, x=3 * MB, x_stride=64, out=4 * MB, out_stride=64)
        a.update(kw)
        return L.expert_dispatch(ctypes.byref(experts._DispatchArgs(**a)), None)
    assert L.expert_dispatch(None, None) == INVALID and call(rows=0, out=None) == OK
    for bad in MOVES_BAD + [dict(x=None), dict(out=None), dict(x=3 * MB + 1), dict(x_stride=63), dict(out_stride=8), dict(out=3 * MB),
                            dict(out=MB), dict(used=2 * MB + 2), dict(out=2 * MB)]:
        assert call(**bad) == INVALID, bad
    assert call(dtype=3) == UNSUPPORTED


def test_combine_refusals(L):
    def call(**kw):
        a = dict(dtype=2, weight_dtype=0, tokens=16, rows=32, choices=2, channels=64, places=MB, weights=2 * MB, y=3 * MB, y_stride=64,
                 out=4 * MB, out_stride=64)
        a.update(kw)
        return L.expert_combine(ctypes.byref(experts._CombineArgs(**a)), None)
    assert L.expert_combine(None, None) == INVALID and call(tokens=0, out=None, places=None) == OK
    for bad in MOVES_BAD + [dict(y=None), dict(out=None), dict(y=3 * MB + 1), dict(y_stride=63), dict(out=3 * MB + 256), dict(out=2 * MB),
                            dict(weights=2 * MB + 2)]:
        assert call(**bad) == INVALID, bad
    assert call(dtype=3) == UNSUPPORTED and call(weight_dtype=1) == UNSUPPORTED


def test_combine_grad_refusals(L):
    def call(**kw):
        a = dict(dtype=2, weight_dtype=2, tokens=16, rows=32, choices=2, channels=64, places=MB, used=2 * MB, weights=3 * MB, dout=4 * MB,
                 dout_stride=64, y=5 * MB, y_stride=64, dy=6 * MB, dy_stride=64, dweights=7 * MB)
        a.update(kw)
        return L.expert_combine_grad(ctypes.byref(experts._CombineGradArgs(**a)), None)
    assert L.expert_combine_grad(None, None) == INVALID
    for bad in MOVES_BAD + [dict(dout=None), dict(dy=None), dict(y=None), dict(y_stride=1), dict(dout_stride=1), dict(dy_stride=1), dict(dy=5 * MB),
                            dict(dy=4 * MB), dict(dweights=3 * MB), dict(dweights=6 * MB), dict(dweights=7 * MB + 2), dict(used=2 * MB + 1)]:
        assert call(**bad) == INVALID, bad
    assert call(dtype=-1) == UNSUPPORTED and call(weight_dtype=1) == UNSUPPORTED


def test_sample_refusals(L):
    def call(**kw):
        a = dict(dtype=0, token_bytes=4, rows=8, n=100, logits=MB, logits_stride=100, uniform=2 * MB, temperature=1.0, top_p=1.0, tokens=3 * MB)
        a.update(kw)
        return L.sample_tokens(ctypes.byref(sampling._SampleArgs(**a)), None)
    assert L.sample_tokens(None, None) == INVALID and call(rows=0, logits=None) == OK
    for bad in (dict(token_bytes=2), dict(n=0), dict(n=(1 << 19) + 1), dict(rows=1 << 31), dict(logits=None), dict(logits=MB + 1), dict(logits_stride=99),
                dict(logits_stride=(1 << 31) + 1), dict(uniform=None), dict(uniform=2 * MB + 1), dict(tokens=None), dict(tokens=3 * MB + 2),
                dict(tokens=MB + 400), dict(tokens=2 * MB), dict(temperatures=MB + 2), dict(top_ks=MB + 1), dict(top_ps=3 * MB), dict(min_ps=3 * MB + 1),
                dict(token_bytes=8, tokens=3 * MB + 4)):
        assert call(**bad) == INVALID, bad
    assert call(dtype=4) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    i, f = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 8)
    plan = dw.ExpertPlan(torch.zeros(5, dtype=torch.int32), i, i.view(-1))
    for bad in (lambda: dw.expert_split(i, 4), lambda: dw.expert_dispatch(f, plan), lambda: dw.expert_combine(f, plan),
                lambda: dw.expert_combine_grad(f, f, plan), lambda: dw.expert_dispatch_grad(f, plan), lambda: dw.sample_tokens(f, f[:, 0])):
        with pytest.raises(ValueError, match="device tensor"):
            bad()
    with pytest.raises(ValueError, match="requires a gradient"):
        dw.sample_tokens(f.requires_grad_(), f[:, 0])


def test_sampling_reference_by_hand():
    z = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))
    at = lambda u, **kw: sr.token(z, u, **kw)[0]  # noqa: E731
    assert [at(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.59, 0.61, 0.89, 0.91, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3, 4, 4]
    # kept: tokens 1 and 3, and of three equal ones the first
    assert [at(u, top_k=3) for u in (0.1, 0.13, 0.6, 0.65, 0.99)] == [0, 1, 1, 3, 3]
    assert [at(u, top_p=0.69) for u in (0.56, 0.58)] == [1, 3] and at(0.99, top_p=0.39) == 1 and at(0.05, top_p=0.75) == 0
    assert [at(u, min_p=0.5) for u in (0.0, 0.56, 0.58)] == [1, 1, 3] and at(0.9, min_p=9.0) == 1
    # top-p is a share of what top-k left: 0.4 / 0.7 reaches 0.57
    assert at(0.99, top_k=2, top_p=0.57) == 1 and at(0.99, top_k=2, top_p=0.58) == 3
    assert at(0.5, temperature=0.0) == 1 and at(0.99, temperature=1e-9) == 1
    assert sr.token(np.full(3, -np.inf), 0.5)[0] == -1 and sr.token(np.array([np.nan, 1.0, -np.inf]), 0.9)[0] == 1
    assert [sr.token(np.array([1.0, np.inf, 2.0, np.inf]), u)[0] for u in (0.4, 0.6)] == [1, 3]
