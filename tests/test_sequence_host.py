"""The sequence operators without a GPU: refusals of the C ABI and of the binding, workspace
sizes, the layout of the argument structures, and the 64-bit reference's gradients against
differences."""
import ctypes
import re
import os

import numpy as np
import pytest
import torch

import device_wide_prefix_tile_amd as dw
import sequence_reference as ref
from device_wide_prefix_tile_amd import sequence as seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = 0, 1, 2
MB = 1 << 20  # fake device addresses, a mebibyte apart: rejected calls never touch them


@pytest.fixture(scope="module")
def L():
    return seq._lib()


# ---------------------------------------------------------------------- layout
@pytest.mark.parametrize("name,cls", [("causal_conv1d_args_t", seq._ConvArgs), ("causal_conv1d_grad_args_t", seq._ConvGradArgs),
                                      ("causal_conv1d_step_args_t", seq._ConvStepArgs), ("selective_scan_args_t", seq._ScanArgs),
                                      ("selective_scan_grad_args_t", seq._ScanGradArgs),
                                      ("selective_scan_step_args_t", seq._ScanStepArgs)])
def test_structures_match_the_header(name, cls):
    text = open(os.path.join(ROOT, "include", "dwpt_seq.h"), encoding="utf-8").read()
    end = text.index("} %s;" % name)
    body = text[text.rindex("typedef struct {", 0, end) + len("typedef struct {"):end]
    fields = []
    for decl in body.split(";"):
        decl = decl.strip()
        if not decl:
            continue
        base, names = re.match(r"((?:const )?\w+)\s*(.*)", decl, re.S).groups()
        for n in names.split(","):
            n = n.strip()
            ctype = (ctypes.c_void_p if n.startswith("*") or "*" in base else
                     {"int32_t": ctypes.c_int32, "uint32_t": ctypes.c_uint32, "uint64_t": ctypes.c_uint64,
                      "int64_t": ctypes.c_int64, "causal_conv1d_args_t": seq._ConvArgs,
                      "selective_scan_args_t": seq._ScanArgs}[base])
            fields.append((n.lstrip("* "), ctype))
    assert [(f[0], f[1]) for f in cls._fields_] == fields


# ---------------------------------------------------------------------- C ABI refusals
def test_embedding_lookup_refusals(L):
    def call(dtype=2, tokens=MB, tb=4, n=8, table=2 * MB, stride=64, v=100, d=64, out=3 * MB):
        return L.embedding_lookup(dtype, tokens, tb, n, table, stride, v, d, 1.0, out, None)
    assert call(n=0, tokens=None, table=None, out=None) == OK  # nothing to do
    assert call(dtype=3) == UNSUPPORTED
    for bad in (dict(tb=2), dict(tokens=None), dict(tokens=MB + 2), dict(table=None), dict(out=None), dict(table=2 * MB + 1),
                dict(stride=63), dict(v=0), dict(v=(1 << 24) + 1), dict(d=0), dict(n=1 << 31), dict(out=2 * MB + 128),
                dict(out=MB), dict(tb=8, tokens=MB + 4)):
        assert call(**bad) == INVALID, bad


def test_embedding_grad_refusals(L):
    need = L.embedding_grad_workspace(8, 100, 64)

    def call(dtype=2, gd=2, tokens=MB, tb=4, n=8, dout=2 * MB, stride=64, v=100, d=64, acc=0, out=3 * MB, ws=4 * MB, wb=need):
        return L.embedding_grad(dtype, gd, tokens, tb, n, dout, stride, v, d, 1.0, acc, out, ws, wb, None)
    assert call(dtype=5) == UNSUPPORTED and call(gd=1) == UNSUPPORTED
    for bad in (dict(ws=None), dict(wb=need - 1), dict(ws=4 * MB + 16), dict(out=None), dict(dout=None), dict(stride=10),
                dict(tokens=None), dict(v=0), dict(d=0), dict(out=2 * MB), dict(ws=3 * MB), dict(n=1 << 31), dict(tb=1)):
        assert call(**bad) == INVALID, bad
    # the workspace grows with the tokens, the table and the channels
    assert L.embedding_grad_workspace(70000, 100, 64) > L.embedding_grad_workspace(65536, 100, 64) > need
    assert L.embedding_grad_workspace(8, 1 << 24, 64) >= 8 << 24
    assert L.embedding_grad_workspace(8, (1 << 24) + 1, 64) == 0


def conv_args(**kw):
    a = dict(dtype=2, weight_dtype=2, activation=1, width=4, rows=32, seqs=2, seq_offsets=None, channels=64, x=MB, x_stride=64,
             weight=2 * MB, bias=3 * MB, initial_state=4 * MB, y=5 * MB, y_stride=64, final_state=6 * MB)
    a.update(kw)
    return seq._ConvArgs(**a)


CONV_BAD = [dict(x=None), dict(x=MB + 1), dict(x_stride=63), dict(weight=None), dict(weight=2 * MB + 1), dict(bias=3 * MB + 1),
            dict(rows=33), dict(seqs=0), dict(rows=1 << 31), dict(channels=0), dict(seq_offsets=MB + 2), dict(initial_state=MB * 4 + 1)]
CONV_UNSUPPORTED = [dict(dtype=9), dict(weight_dtype=1), dict(width=1), dict(width=5), dict(activation=2)]


def test_conv_refusals(L):
    call = lambda **kw: L.causal_conv1d(ctypes.byref(conv_args(**kw)), None)  # noqa: E731
    assert L.causal_conv1d(None, None) == INVALID
    for bad in CONV_BAD + [dict(y=None), dict(y_stride=1), dict(y=MB), dict(y=MB + 64), dict(final_state=4 * MB), dict(final_state=5 * MB)]:
        assert call(**bad) == INVALID, bad
    for bad in CONV_UNSUPPORTED:
        assert call(**bad) == UNSUPPORTED, bad
    # rows of one stride side by side are not an overlap, crossing ones are
    assert call(x_stride=128, y=MB + 2 * 32, y_stride=128) == INVALID


def test_conv_grad_refusals(L):
    need = L.causal_conv1d_grad_workspace(ctypes.byref(conv_args()))
    assert need > 0

    def call(fwd=(), **kw):
        g = dict(args=conv_args(**dict(fwd)), dy=8 * MB, dy_stride=64, dfinal_state=9 * MB, dx=10 * MB, dx_stride=64,
                 dweight=11 * MB, dbias=12 * MB, dinitial_state=13 * MB, workspace=14 * MB, workspace_bytes=need)
        g.update(kw)
        return L.causal_conv1d_grad(ctypes.byref(seq._ConvGradArgs(**g)), None)
    assert L.causal_conv1d_grad(None, None) == INVALID
    for bad in CONV_BAD:
        assert call(fwd=bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dx=None), dict(dx=8 * MB), dict(dweight=None), dict(workspace=None), dict(workspace_bytes=need - 1),
                dict(workspace=14 * MB + 8), dict(dx_stride=2), dict(dinitial_state=4 * MB), dict(dbias=11 * MB)):
        assert call(**bad) == INVALID, bad


def test_conv_step_refusals(L):
    def call(**kw):
        a = dict(dtype=2, weight_dtype=0, activation=0, width=3, rows=4, n_slots=9, slots=MB, channels=64, x=2 * MB, x_stride=64,
                 weight=3 * MB, bias=None, state=4 * MB, y=5 * MB, y_stride=64)
        a.update(kw)
        return L.causal_conv1d_step(ctypes.byref(seq._ConvStepArgs(**a)), None)
    assert call(rows=0, x=None, y=None) == OK
    for bad in (dict(x=None), dict(y=None), dict(state=None), dict(weight=None), dict(rows=65536), dict(y=2 * MB), dict(state=2 * MB),
                dict(x_stride=1), dict(slots=MB + 1), dict(channels=0), dict(n_slots=1 << 31)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(width=5), dict(dtype=4), dict(weight_dtype=1), dict(activation=-1)):
        assert call(**bad) == UNSUPPORTED, bad


def scan_args(**kw):
    a = dict(dtype=2, delta_softplus=1, rows=32, seqs=2, channels=64, states=16, groups=2, x=MB, x_stride=64, delta=2 * MB,
             delta_stride=64, A=3 * MB, B=4 * MB, b_stride=32, C=5 * MB, c_stride=32, D=6 * MB, z=7 * MB, z_stride=64,
             delta_bias=8 * MB, initial_state=9 * MB, y=10 * MB, y_stride=64, final_state=11 * MB, saved=12 * MB,
             workspace=13 * MB, workspace_bytes=MB)
    a.update(kw)
    return seq._ScanArgs(**a)


SCAN_BAD = [dict(x=None), dict(delta=None), dict(A=None), dict(B=None), dict(C=None), dict(x=MB + 1), dict(z=7 * MB + 1), dict(b_stride=31),
            dict(c_stride=16), dict(groups=3), dict(groups=0), dict(channels=0), dict(rows=33), dict(seqs=0), dict(rows=1 << 31),
            dict(A=3 * MB + 2), dict(D=6 * MB + 1), dict(delta_bias=8 * MB + 2), dict(saved=12 * MB + 4), dict(seq_offsets=MB + 1)]
SCAN_UNSUPPORTED = [dict(states=0), dict(states=65), dict(dtype=-1)]


def test_scan_refusals(L):
    call = lambda **kw: L.selective_scan(ctypes.byref(scan_args(**kw)), None)  # noqa: E731
    assert L.selective_scan(None, None) == INVALID
    for bad in SCAN_BAD + [dict(y=MB), dict(y=10 * MB + 1), dict(y_stride=3), dict(workspace=None), dict(workspace_bytes=1),
                           dict(workspace=13 * MB + 4), dict(final_state=9 * MB), dict(saved=10 * MB), dict(workspace=MB)]:
        assert call(**bad) == INVALID, bad
    for bad in SCAN_UNSUPPORTED:
        assert call(**bad) == UNSUPPORTED, bad


def test_scan_grad_refusals(L):
    def call(fwd=(), **kw):
        g = dict(args=scan_args(**dict(fwd)), dy=20 * MB, dy_stride=64, dfinal_state=21 * MB, dx=22 * MB, dx_stride=64,
                 ddelta=23 * MB, ddelta_stride=64, dz=24 * MB, dz_stride=64, dB=25 * MB, db_stride=32, dC=26 * MB, dc_stride=32,
                 dA=27 * MB, dD=28 * MB, ddelta_bias=29 * MB, dinitial_state=30 * MB)
        g.update(kw)
        return L.selective_scan_grad(ctypes.byref(seq._ScanGradArgs(**g)), None)
    assert L.selective_scan_grad(None, None) == INVALID
    for bad in SCAN_BAD + [dict(saved=None), dict(workspace=None), dict(workspace_bytes=256), dict(z=None), dict(D=None), dict(delta_bias=None)]:
        assert call(fwd=bad) == INVALID, bad
    for bad in (dict(dy=None), dict(dx=None), dict(ddelta=None), dict(dz=None), dict(dB=None), dict(dC=None), dict(dA=None), dict(dD=None),
                dict(ddelta_bias=None), dict(dx=20 * MB), dict(dB=26 * MB), dict(db_stride=3), dict(dx=MB), dict(dinitial_state=21 * MB)):
        assert call(**bad) == INVALID, bad


def test_scan_step_refusals(L):
    def call(**kw):
        a = dict(dtype=0, rows=4, n_slots=9, slots=MB, channels=64, states=16, groups=1, x=2 * MB, x_stride=64, delta=3 * MB,
                 delta_stride=64, A=4 * MB, B=5 * MB, b_stride=16, C=6 * MB, c_stride=16, state=7 * MB, y=8 * MB, y_stride=64)
        a.update(kw)
        return L.selective_scan_step(ctypes.byref(seq._ScanStepArgs(**a)), None)
    assert call(rows=0) == OK
    for bad in (dict(x=None), dict(delta=None), dict(A=None), dict(B=None), dict(C=None), dict(state=None), dict(y=None), dict(y=2 * MB),
                dict(state=8 * MB), dict(groups=5), dict(y_stride=1), dict(state=7 * MB + 2), dict(n_slots=1 << 31), dict(slots=MB + 2)):
        assert call(**bad) == INVALID, bad
    assert call(states=65) == UNSUPPORTED and call(dtype=7) == UNSUPPORTED


def test_workspace_queries_follow_the_plan(L):
    """Enough sequences and channels need no spans; one long sequence is cut into some."""
    wide = dict(groups=1, x_stride=4096, delta_stride=4096, z_stride=4096, y_stride=4096)
    many = scan_args(rows=64 * 256, seqs=64, channels=4096, **wide)
    one = scan_args(rows=64 * 256, seqs=1, channels=256, **wide)
    assert L.selective_scan_workspace(ctypes.byref(many)) == 256
    assert L.selective_scan_workspace(ctypes.byref(one)) > 256 * 16 * 4
    # the saved states: one per 16 rows, channel and (padded) state
    assert L.selective_scan_saved(ctypes.byref(many)) == 64 * 16 * 4096 * 16
    assert L.selective_scan_saved(ctypes.byref(scan_args(rows=0, seqs=0, x=None, delta=None, B=None, C=None, z=None, y=None))) == 0
    assert L.selective_scan_workspace(ctypes.byref(scan_args(groups=3))) == 0


# ---------------------------------------------------------------------- binding refusals
def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        dw.causal_conv1d(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        dw.selective_scan(x, x, torch.zeros(8, 4), torch.zeros(1, 4, 1, 4), torch.zeros(1, 4, 1, 4))
    with pytest.raises(ValueError):
        dw.embedding_lookup(torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        dw.embedding_lookup(torch.zeros(3), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        dw.causal_conv1d(x.double(), torch.zeros(8, 4).double())


def test_row_strides():
    rows = seq._rows
    wide = torch.zeros(3, 5, 24)
    assert rows(wide, "t") == 24 and rows(wide[..., 8:16], "t") == 24
    assert rows(torch.zeros(7, 8)[::2], "t") == 16
    assert rows(torch.zeros(4, 1, 8), "t") == 8 and rows(torch.zeros(4, 2, 8)[:, :1], "t") == 16
    assert rows(torch.zeros(6, 2, 4), "t", inner=2) == 8
    assert rows(torch.zeros(2, 3, 32)[..., :16].unflatten(-1, (2, 8)), "t", inner=2) == 32
    assert rows(torch.zeros(0, 8), "t") >= 8
    for bad in (wide.transpose(1, 2), wide[:, :4], wide[..., ::2], torch.zeros(1, 8).expand(5, 8), torch.zeros(5, 8).t()):
        with pytest.raises(ValueError):
            rows(bad, "t")


# ---------------------------------------------------------------------- the reference against differences
def directional(f, args, name, rng, h=1e-6):
    """(change of f along a random direction of args[name] per unit, direction)"""
    v = rng.standard_normal(args[name].shape)
    up, down = dict(args), dict(args)
    up[name], down[name] = args[name] + h * v, args[name] - h * v
    return (f(**up) - f(**down)) / (2 * h), v


def test_reference_scan_gradients_match_differences():
    rng = np.random.default_rng(5)
    rows, d, g, n = 11, 6, 2, 3
    seqs = [(0, 4), (4, 4), (4, 5), (5, 11)]
    args = dict(x=rng.standard_normal((rows, d)), delta=rng.standard_normal((rows, d)), A=-rng.uniform(0.3, 2, (d, n)),
                B=rng.standard_normal((rows, g, n)), C=rng.standard_normal((rows, g, n)), D=rng.standard_normal(d),
                z=rng.standard_normal((rows, d)), bias=rng.standard_normal(d), initial=rng.standard_normal((4, d, n)))
    dy, dfin = rng.standard_normal((rows, d)), rng.standard_normal((4, d, n))

    def loss(**kw):
        r = ref.scan(sp=True, seqs=seqs, **kw)
        return (r["y"][0] * dy).sum() + (r["final"][0] * dfin).sum()
    grads = ref.scan(sp=True, seqs=seqs, dy=dy, dfinal=dfin, **args)
    for name, of in (("x", "dx"), ("delta", "ddelta"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                     ("bias", "ddelta_bias"), ("initial", "dinitial")):
        got, v = directional(loss, args, name, rng)
        want = (grads[of][0] * v).sum()
        # central differences: h^2 of the third derivative, and 2^-52 / h of the loss's terms
        assert abs(got - want) <= 1e-7 * (1 + np.abs(grads[of][0] * v).sum()), name


def test_reference_conv_gradients_match_differences():
    rng = np.random.default_rng(6)
    rows, d, k = 9, 5, 4
    seqs = [(0, 2), (2, 2), (2, 8), (8, 9)]
    args = dict(x=rng.standard_normal((rows, d)), w=rng.standard_normal((d, k)), b=rng.standard_normal(d),
                initial=rng.standard_normal((4, k - 1, d)))
    dy, dfin = rng.standard_normal((rows, d)), rng.standard_normal((4, k - 1, d))

    def loss(**kw):
        r = ref.conv(act=True, seqs=seqs, **kw)
        return (r["y"][0] * dy).sum() + (r["final"][0] * dfin).sum()
    grads = ref.conv(act=True, seqs=seqs, dy=dy, dfinal=dfin, **args)
    for name, of in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("initial", "dinitial")):
        got, v = directional(loss, args, name, rng)
        want = (grads[of][0] * v).sum()
        assert abs(got - want) <= 1e-7 * (1 + np.abs(grads[of][0] * v).sum()), name
