"""Tokens sorted by expert and back over torch tensors: the stable split of every token's choices by
expert, the tokens' rows in the experts' order, the experts' results added up again with weights
applied, and the gradients (C ABI in include/dwpt_seq.h).

As in ``sequence``: every step runs in the library's HIP kernels on the current stream of the tensors'
device (or on ``stream``), nothing synchronises, nothing is recorded for autograd.

    plan = expert_split(experts, n_experts)           # experts (n, k) int32: a router's choices
    rows = expert_dispatch(x, plan)                   # expert e has rows[plan.offsets[e]:plan.offsets[e + 1]]
    ...                                               # y: the experts' results, row by row
    out = expert_combine(y, plan, weights)            # weights (n, k)
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .sequence import (_DTYPE, _I, _I64, _P, _U32, _U64, _check, _enqueue, _lib, _like, _no_graph, _plain, _ptr, _register, _rows, _x)


class _DispatchArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("clear", _I), ("tokens", _U64), ("rows", _U64), ("choices", _U32), ("channels", _U32),
                ("places", _P), ("used", _P), ("x", _P), ("x_stride", _I64), ("out", _P), ("out_stride", _I64), ("source", _P),
                ("source_rows", _U64)]


class _CombineArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("weight_dtype", _I), ("tokens", _U64), ("rows", _U64), ("choices", _U32), ("channels", _U32),
                ("places", _P), ("weights", _P), ("y", _P), ("y_stride", _I64), ("out", _P), ("out_stride", _I64)]


class _CombineGradArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("weight_dtype", _I), ("tokens", _U64), ("rows", _U64), ("choices", _U32), ("channels", _U32),
                ("places", _P), ("used", _P), ("weights", _P), ("dout", _P), ("dout_stride", _I64), ("y", _P), ("y_stride", _I64),
                ("dy", _P), ("dy_stride", _I64), ("dweights", _P), ("source", _P), ("source_rows", _U64), ("clear", _I), ("reserved", _I)]


_register({
    "expert_split": ([_P, _U64, _U32, _P, _P, _P, _P, _U64, _P], _I),
    "expert_split_workspace": ([_U64, _U32], _U64),
    "expert_dispatch": ([ctypes.POINTER(_DispatchArgs), _P], _I),
    "expert_combine": ([ctypes.POINTER(_CombineArgs), _P], _I),
    "expert_combine_grad": ([ctypes.POINTER(_CombineGradArgs), _P], _I),
})


class ExpertPlan(NamedTuple):
    """Which choice has which row.  offsets (E + 1): expert e has rows offsets[e] .. offsets[e + 1] - 1 of the experts'
    order; places (n, k): the row of every choice, -1 for a choice of no expert; source (n k): the choice t k + j
    of every row, -1 from row offsets[E] on.  All int32."""
    offsets: torch.Tensor
    places: torch.Tensor
    source: torch.Tensor


class CombineGrads(NamedTuple):
    """Gradients of expert_combine; dweights is float32, and None without weights."""
    dy: torch.Tensor
    dweights: Optional[torch.Tensor]


def expert_split(experts: torch.Tensor, n_experts: int, stream=None) -> ExpertPlan:
    """The stable split of the choices by expert: every expert's rows hold its choices in the order t k + j.

    experts: (n, k) int32, contiguous; a number outside 0 .. n_experts - 1 is a choice of no expert (padding, a token
    that is dropped).  n_experts <= 1024."""
    _no_graph(experts, "experts")
    if experts.dtype != torch.int32 or experts.dim() != 2 or experts.shape[1] < 1:
        raise TypeError("experts must be an (n, k) int32 tensor")
    if not experts.is_cuda or not experts.is_contiguous():
        raise ValueError("experts must be a contiguous device tensor")
    if not 1 <= n_experts <= 1024:
        raise ValueError("n_experts must be in 1 .. 1024")
    n = experts.numel()

    def call(handle):
        L = _lib()
        need = L.expert_split_workspace(n, n_experts)
        new = experts.new_empty
        offsets, places, source = new(n_experts + 1), new(experts.shape), new(n)
        ws = new((need + 3) // 4) if need else None
        _check(L.expert_split(experts.data_ptr(), n, n_experts, offsets.data_ptr(), places.data_ptr(), source.data_ptr(), _ptr(ws), need,
                              handle), "expert_split")
        return ExpertPlan(offsets, places, source)

    return _enqueue(experts, stream, call)


def _plan(plan: ExpertPlan, device: int):
    """(tokens, choices, address of places)"""
    places, offsets = plan.places, plan.offsets
    if places.dim() != 2 or not 1 <= places.shape[1] <= 256:
        raise ValueError("plan.places must be (n, k) with k in 1 .. 256")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("plan.offsets must be (E + 1,)")
    at = _plain(places, "plan.places", places.shape, torch.int32, device)
    _plain(offsets, "plan.offsets", offsets.shape, torch.int32, device)
    return places.shape[0], places.shape[1], at


def _source(plan: ExpertPlan, device: int):
    """(address, values) of a plan's source, which only says where nothing need be cleared: (None, 0) for one that is not as
    expert_split makes it."""
    s = plan.source
    if not isinstance(s, torch.Tensor) or s.dtype != torch.int32 or s.get_device() != device or not s.is_contiguous():
        return None, 0
    return s.data_ptr(), s.numel()


def _matrix(t: torch.Tensor, name: str, rows=None):
    _x(t, name)
    if t.dim() != 2 or t.shape[1] < 1 or (rows is not None and t.shape[0] != rows):
        raise ValueError("%s must be (%s, D)" % (name, "rows" if rows is None else rows))
    return t.shape[1]


def _result(out, shape, like: torch.Tensor, name: str):
    """(tensor, address, row stride) of an output of that shape: `out`, or a new one."""
    if out is None:
        out = like.new_empty(shape)
        return out, out.data_ptr(), shape[1]
    return (out,) + _like(out, name, torch.Size(shape), like.dtype, like.get_device(), shape[1])


def expert_dispatch(x: torch.Tensor, plan: ExpertPlan, out: Optional[torch.Tensor] = None, stream=None):
    """The tokens' rows in the experts' order: out[plan.places[t, j]] = x[t].

    x: (n, D), any row stride.  A new out is (n k, D), its rows that no place leads to zero; in a given one (rows, D) they
    are left as they were, and places outside it are skipped.  Places may be taken out of a plan (-1) after the split."""
    d = _matrix(x, "x", plan.places.shape[0])
    n, k, places = _plan(plan, x.get_device())
    source = _source(plan, x.get_device()) if out is None else (None, 0)

    def call(handle):
        y, to, stride = _result(out, (n * k, d), x, "out") if out is None else _result(out, (out.shape[0], d), x, "out")
        a = _DispatchArgs(_DTYPE[x.dtype], 1 if out is None else 0, n, y.shape[0], k, d, places, None, x.data_ptr(), _rows(x, "x"), to,
                          stride, *source)
        _check(_lib().expert_dispatch(ctypes.byref(a), handle), "expert_dispatch")
        return y

    return _enqueue(x, stream, call)


def _combine(y, plan, weights, out, stream, what, name):
    d = _matrix(y, name)
    n, k, places = _plan(plan, y.get_device())
    w = _weights(weights, plan, y)

    def call(handle):
        o, to, stride = _result(out, (n, d), y, "dx" if what == "expert_dispatch_grad" else "out")
        a = _CombineArgs(_DTYPE[y.dtype], 0 if weights is None else _DTYPE[weights.dtype], n, y.shape[0], k, d, places, w, y.data_ptr(),
                         _rows(y, name), to, stride)
        _check(_lib().expert_combine(ctypes.byref(a), handle), what)
        return o

    return _enqueue(y, stream, call)


def _weights(weights, plan: ExpertPlan, y: torch.Tensor):
    """Address of the weights, or None."""
    if weights is None:
        return None
    if weights.dtype != y.dtype and weights.dtype != torch.float32:
        raise TypeError("weights must be of the rows' type or float32")
    return _plain(weights, "weights", plan.places.shape, weights.dtype, y.get_device())


def expert_dispatch_grad(drows: torch.Tensor, plan: ExpertPlan, dx: Optional[torch.Tensor] = None, stream=None):
    """Gradient of ``expert_dispatch`` by x: dx[t] = the sum over j of drows[plan.places[t, j]], added up in 32 bits."""
    return _combine(drows, plan, None, dx, stream, "expert_dispatch_grad", "drows")


def expert_combine(y: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                   stream=None):
    """The rows of every token added up: out[t] = sum over j of weights[t, j] y[plan.places[t, j]], in 32 bits and in the
    order of j; a choice of no expert adds nothing.

    y: (rows, D), any row stride; weights: (n, k) of y's type or float32, contiguous (None: ones)."""
    return _combine(y, plan, weights, out, stream, "expert_combine", "y")


def expert_combine_grad(dout: torch.Tensor, y: torch.Tensor, plan: ExpertPlan, weights: Optional[torch.Tensor] = None,
                        dy: Optional[torch.Tensor] = None, stream=None) -> CombineGrads:
    """Gradients of ``expert_combine`` (its arguments) for dout (n, D): dy[plan.places[t, j]] = weights[t, j] dout[t], and
    dweights[t, j] = the sum over the channels of dout[t] y[plan.places[t, j]].

    dy may be given to write into; its rows that no place leads to are left as they were then, and are zero otherwise."""
    d = _matrix(dout, "dout", plan.places.shape[0])
    n, k, places = _plan(plan, dout.get_device())
    source = _source(plan, dout.get_device()) if dy is None else (None, 0)
    _matrix(y, "y")
    y_at, y_stride = _like(y, "y", torch.Size((y.shape[0], d)), dout.dtype, dout.get_device(), d)
    w = _weights(weights, plan, dout)

    def call(handle):
        o, to, stride = _result(dy, (y.shape[0], d), dout, "dy")
        dw = None if weights is None else torch.empty(plan.places.shape, dtype=torch.float32, device=dout.device)
        a = _CombineGradArgs(_DTYPE[dout.dtype], 0 if weights is None else _DTYPE[weights.dtype], n, y.shape[0], k, d, places,
                             None, w, dout.data_ptr(), _rows(dout, "dout"), y_at, y_stride, to, stride,
                             None if dw is None else dw.data_ptr(), *source, 1 if dy is None else 0)
        _check(_lib().expert_combine_grad(ctypes.byref(a), handle), "expert_combine_grad")
        return CombineGrads(o, dw)

    return _enqueue(dout, stream, call)
