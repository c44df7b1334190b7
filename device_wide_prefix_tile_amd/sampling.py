"""Sampling of tokens over torch tensors: temperature, top-k, top-p and min-p from given random numbers
(C ABI in include/dwpt_seq.h).  As in ``sequence``, one kernel on the current stream of the tensors' device."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from .sequence import _DTYPE, _I, _I64, _P, _U32, _U64, _check, _enqueue, _lib, _plain, _register, _rows, _x

_F64 = ctypes.c_double


class _SampleArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("token_bytes", _I), ("rows", _U64), ("n", _U32), ("reserved", _U32), ("logits", _P),
                ("logits_stride", _I64), ("uniform", _P), ("temperatures", _P), ("top_ks", _P), ("top_ps", _P), ("min_ps", _P),
                ("temperature", _F64), ("top_p", _F64), ("min_p", _F64), ("top_k", _I64), ("tokens", _P)]


_register({"sample_tokens": ([ctypes.POINTER(_SampleArgs), _P], _I)})


def _setting(value, name: str, rows: int, dtype, device: int):
    """(address of the rows' values or None, value for all rows)"""
    if isinstance(value, torch.Tensor):
        return _plain(value, name, (rows,), dtype, device), 0
    return None, value


def sample_tokens(logits: torch.Tensor, uniform: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
                  out: Optional[torch.Tensor] = None, stream=None):
    """One token for every row of logits (rows, V), V <= 2^19, from uniform (rows,) float32 in [0, 1).

    Weights w = exp((logit - max) / temperature), of which are kept, by falling logit (equal ones by ascending
    index): the first top_k (0: all), of these the first whose predecessors add up to less than top_p of their sum (at
    least one), and those with w >= min_p.  The token is the first kept one, by index, up to which the kept weights
    exceed uniform times their sum.  A temperature of 0 takes the first largest logit.  Logits of minus infinity and NaN
    are never taken; a row of nothing else gives -1.

    temperature, top_p, min_p: numbers, or (rows,) float32; top_k: a number, or (rows,) int32.  out: (rows,) int32 or
    int64 to write into; a new one is int32."""
    _x(logits, "logits")
    if logits.dim() != 2 or not 1 <= logits.shape[1] <= 1 << 19:
        raise ValueError("logits must be (rows, V) with V in 1 .. 2^19")
    rows, n = logits.shape
    device = logits.get_device()
    u = _plain(uniform, "uniform", (rows,), torch.float32, device)
    ts, t = _setting(temperature, "temperature", rows, torch.float32, device)
    ks, k = _setting(top_k, "top_k", rows, torch.int32, device)
    ps, p = _setting(top_p, "top_p", rows, torch.float32, device)
    ms, m = _setting(min_p, "min_p", rows, torch.float32, device)
    stride = _rows(logits, "logits")
    if out is not None and out.dtype not in (torch.int32, torch.int64):
        raise TypeError("out must be int32 or int64")

    def call(handle):
        y = uniform.new_empty(rows, dtype=torch.int32) if out is None else out
        to = _plain(y, "out", (rows,), y.dtype, device)
        a = _SampleArgs(_DTYPE[logits.dtype], y.element_size(), rows, n, 0, logits.data_ptr(), stride, u, ts, ks, ps, ms, t, p, m, k, to)
        _check(_lib().sample_tokens(ctypes.byref(a), handle), "sample_tokens")
        return y

    return _enqueue(logits, stream, call)
