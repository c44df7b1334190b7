"""Sequence-model operators over torch tensors: embedding lookup and its gradient by sorted
tokens, the short causal convolution and the selective state-space scan, with their gradients
and their single-token forms (C ABI in include/dwpt_seq.h).

Argument marshalling only, as in ``binding``: every step runs in the library's HIP kernels, calls
enqueue on the current stream of the tensors' device (or on ``stream``) and return without
synchronising, and there is no CPU fallback.  Outputs and workspaces come from torch's allocator
on the stream that the call runs on, so a call can be captured into a graph.

The gradients are functions of their own: nothing is recorded for autograd.  Where autograd is
recording, a tensor that requires a gradient is refused rather than detached without a word; call
under ``torch.no_grad()``, inside an ``autograd.Function``, or with ``tensor.detach()``.

Layout: channels last.  Rows are (B, L, D) for B sequences of one length, or (rows, D) with
``seq_offsets`` (int32, S + 1 ascending) for sequences packed one behind the other.  A tensor of
rows may be a slice of a wider one (any row stride); its last dimension is contiguous.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from .binding import ScanError, _raw_stream, lib

_DTYPE = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_ACT = {None: 0, "silu": 1}
_P, _I, _I64, _U32, _U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_uint64


class _ConvArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("weight_dtype", _I), ("activation", _I), ("width", _I), ("rows", _U64), ("seqs", _U64),
                ("seq_offsets", _P), ("channels", _U32), ("reserved", _U32), ("x", _P), ("x_stride", _I64), ("weight", _P),
                ("bias", _P), ("initial_state", _P), ("y", _P), ("y_stride", _I64), ("final_state", _P)]


class _ConvGradArgs(ctypes.Structure):
    _fields_ = [("args", _ConvArgs), ("dy", _P), ("dy_stride", _I64), ("dfinal_state", _P), ("dx", _P), ("dx_stride", _I64),
                ("dweight", _P), ("dbias", _P), ("dinitial_state", _P), ("workspace", _P), ("workspace_bytes", _U64)]


class _ConvStepArgs(ctypes.Structure):
    _fields_ = [("dtype", _I), ("weight_dtype", _I), ("activation", _I), ("width", _I), ("rows", _U64), ("n_slots", _U64),
                ("slots", _P), ("channels", _U32), ("reserved", _U32), ("x", _P), ("x_stride", _I64), ("weight", _P),
                ("bias", _P), ("state", _P), ("y", _P), ("y_stride", _I64)]


_SCAN_INPUTS = [("channels", _U32), ("states", _U32), ("groups", _U32), ("reserved", _U32), ("x", _P), ("x_stride", _I64),
                ("delta", _P), ("delta_stride", _I64), ("A", _P), ("B", _P), ("b_stride", _I64), ("C", _P),
                ("c_stride", _I64), ("D", _P), ("z", _P), ("z_stride", _I64), ("delta_bias", _P)]


class _ScanArgs(ctypes.Structure):
    _fields_ = ([("dtype", _I), ("delta_softplus", _I), ("rows", _U64), ("seqs", _U64), ("seq_offsets", _P)] + _SCAN_INPUTS
                + [("initial_state", _P), ("y", _P), ("y_stride", _I64), ("final_state", _P), ("saved", _P),
                   ("workspace", _P), ("workspace_bytes", _U64)])


class _ScanGradArgs(ctypes.Structure):
    _fields_ = [("args", _ScanArgs), ("dy", _P), ("dy_stride", _I64), ("dfinal_state", _P), ("dx", _P), ("dx_stride", _I64),
                ("ddelta", _P), ("ddelta_stride", _I64), ("dz", _P), ("dz_stride", _I64), ("dB", _P), ("db_stride", _I64),
                ("dC", _P), ("dc_stride", _I64), ("dA", _P), ("dD", _P), ("ddelta_bias", _P), ("dinitial_state", _P)]


class _ScanStepArgs(ctypes.Structure):
    _fields_ = ([("dtype", _I), ("delta_softplus", _I), ("rows", _U64), ("n_slots", _U64), ("slots", _P)] + _SCAN_INPUTS
                + [("state", _P), ("y", _P), ("y_stride", _I64)])


SIGNATURES = {
    "embedding_lookup": ([_I, _P, _I, _U64, _P, _I64, _U64, _U32, ctypes.c_float, _P, _P], _I),
    "embedding_grad": ([_I, _I, _P, _I, _U64, _P, _I64, _U64, _U32, ctypes.c_float, _I, _P, _P, _U64, _P], _I),
    "embedding_grad_workspace": ([_U64, _U64, _U32], _U64),
    "causal_conv1d": ([ctypes.POINTER(_ConvArgs), _P], _I),
    "causal_conv1d_grad": ([ctypes.POINTER(_ConvGradArgs), _P], _I),
    "causal_conv1d_grad_workspace": ([ctypes.POINTER(_ConvArgs)], _U64),
    "causal_conv1d_step": ([ctypes.POINTER(_ConvStepArgs), _P], _I),
    "selective_scan": ([ctypes.POINTER(_ScanArgs), _P], _I),
    "selective_scan_workspace": ([ctypes.POINTER(_ScanArgs)], _U64),
    "selective_scan_saved": ([ctypes.POINTER(_ScanArgs)], _U64),
    "selective_scan_grad": ([ctypes.POINTER(_ScanGradArgs), _P], _I),
    "selective_scan_grad_workspace": ([ctypes.POINTER(_ScanGradArgs)], _U64),
    "selective_scan_step": ([ctypes.POINTER(_ScanStepArgs), _P], _I),
}

_seq_lib = None


def _lib():
    global _seq_lib
    if _seq_lib is None:
        L = lib()
        for name, (argtypes, restype) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = argtypes
            fn.restype = restype
        _seq_lib = L
    return _seq_lib


# ---------------------------------------------------------------------- calls
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(x: torch.Tensor, stream, call):
    """call(handle) with x's device current, on the stream asked for: torch allocates on that
    stream inside, so memory that is let go is reused in its order."""
    index = x.get_device()
    if stream is None and _raw_stream is not None and _current_device() == index:
        return call(_raw_stream(index))  # the usual case, without context managers
    with torch.cuda.device(index):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            handle = int(stream)
            if handle == 0:
                stream = torch.cuda.default_stream()
            else:
                stream = torch.cuda.ExternalStream(handle)
        elif stream.device.index != index:
            raise ValueError("stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _check(status: int, what: str):
    if status != 0:
        raise ScanError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(x: torch.Tensor, name: str, t: torch.Tensor):
    if t.get_device() != x.get_device():
        raise ValueError("%s must be on the device of the other tensors" % name)


_recording = torch.is_grad_enabled


def _no_graph(t: torch.Tensor, name: str):
    """Refuses t if autograd would have to record what is done with it."""
    if t.requires_grad and _recording():
        raise ValueError("%s requires a gradient, which the sequence operators do not record: call them under torch.no_grad(), "
                         "or with %s.detach()" % (name, name))


def _refuse(t: torch.Tensor, name: str, shape, dtype):
    """What is wrong with t, which was to have that shape and type, lie on the other tensors' device and need no graph."""
    _no_graph(t, name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    raise ValueError("%s must be on the device of the other tensors" % name)


def _rows(t: torch.Tensor, name: str, inner: int = 1):
    """Row stride of t, whose last `inner` dimensions are contiguous and whose leading ones are one flat run of rows."""
    size = t.shape
    if t.is_contiguous():
        return size[-1] if inner == 1 else size[-1] * size[-2]
    st = t.stride()
    n = len(size)
    if n == 2 and inner == 1 and st[1] == 1 and st[0] >= size[1]:  # a slice of wider rows
        return st[0]
    width = 1
    for k in range(n - 1, n - 1 - inner, -1):
        if size[k] != 1 and st[k] != width:
            raise ValueError("the last dimension%s of %s must be contiguous" % ("s" if inner > 1 else "", name))
        width *= size[k]
    lead = n - inner
    if lead == 0:
        return width
    row = st[lead - 1]
    if size[lead - 1] <= 1:  # one row per sequence (or none): the sequences' stride is the rows'
        if lead == 1 or size[0] <= 1:
            return width if row < width else row
        row = st[0]
    elif lead == 2 and size[0] > 1 and st[0] != size[1] * row:
        raise ValueError("the rows of %s must follow one another at one stride" % name)
    if row < width and t.numel():
        raise ValueError("the rows of %s overlap" % name)
    return max(row, width)


def _plain(t: torch.Tensor, name: str, shape, dtype, device: int):
    """Address of t, a contiguous tensor of that shape, type and device (its index; -1: the host); None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or t.get_device() != device or (t.requires_grad and _recording()):
        _refuse(t, name, shape, dtype)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _like(t: torch.Tensor, name: str, shape, dtype, device: int, width: int, inner: int = 1):
    """(address, row stride) of t, rows of `width` values in that shape, type and device; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.shape != shape or t.dtype != dtype or t.get_device() != device or (t.requires_grad and _recording()):
        _refuse(t, name, shape, dtype)
    return t.data_ptr(), width if t.is_contiguous() else _rows(t, name, inner)


def _x(x: torch.Tensor, name: str = "x"):
    if x.dtype not in _DTYPE:
        raise TypeError("%s must be float32, float16 or bfloat16" % name)
    _no_graph(x, name)
    if not x.is_cuda:
        raise ValueError("%s must be a device tensor" % name)


def _lengths(x: torch.Tensor, seq_offsets):
    """(rows, sequences, offsets pointer)"""
    if seq_offsets is None:
        if x.dim() != 3:
            raise ValueError("x must be (B, L, D), or (rows, D) with seq_offsets")
        return x.shape[0] * x.shape[1], x.shape[0], None
    if x.dim() != 2:
        raise ValueError("with seq_offsets x must be (rows, D)")
    if seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1 or not seq_offsets.is_contiguous() or seq_offsets.shape[0] < 1:
        raise TypeError("seq_offsets must be a contiguous 1-D int32 tensor of S + 1 values")
    _on(x, "seq_offsets", seq_offsets)
    return x.shape[0], seq_offsets.shape[0] - 1, seq_offsets.data_ptr()


def _new_rows(seq_offsets):
    """What makes a new tensor for gradients of rows: the kernels write the rows of sequences, and the gradient
    of a row that belongs to none is zero."""
    return torch.empty if seq_offsets is None else torch.zeros


def _out(out, x: torch.Tensor, name: str, new=torch.empty):
    """(tensor, address, row stride) of an output shaped like x: `out`, or a new one."""
    if out is None:
        out = new(x.shape, dtype=x.dtype, device=x.device)
        return out, out.data_ptr(), x.shape[-1]
    return (out,) + _like(out, name, x.shape, x.dtype, x.get_device(), x.shape[-1])


def _optional_state(state, name: str, shape, dtype, x: torch.Tensor):
    """(tensor, address) of an output state: `state` may be a tensor to write into, or True for a new one."""
    if state is None or state is False:
        return None, None
    if state is True:
        state = torch.empty(shape, dtype=dtype, device=x.device)
        return state, state.data_ptr()
    return state, _plain(state, name, shape, dtype, x.get_device())


# ---------------------------------------------------------------------- embedding
def _tokens(tokens: torch.Tensor):
    if tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError("tokens must be int32 or int64")
    if not tokens.is_cuda or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous device tensor")
    return tokens.element_size()


def embedding_lookup(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                     stream=None):
    """out[..., :] = scale * table[tokens[...]]; a token outside the table gives a row of zeros.

    tokens: int32 or int64 of any shape; table: (V, D) float32, float16 or bfloat16."""
    size = _tokens(tokens)
    _x(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be (V, D)")
    v, d = table.shape
    if v < 1 or d < 1:
        raise ValueError("table must be (V, D)")
    _on(tokens, "table", table)
    stride = _rows(table, "table")
    shape = tokens.shape + (d,)

    def call(handle):
        if out is None:
            y = torch.empty(shape, dtype=table.dtype, device=table.device)
            to = y.data_ptr()
        else:
            y = out
            to = _plain(y, "out", shape, table.dtype, table.get_device())
        _check(_lib().embedding_lookup(_DTYPE[table.dtype], tokens.data_ptr(), size, tokens.numel(), table.data_ptr(), stride,
                                       v, d, scale, to, handle), "embedding_lookup")
        return y

    return _enqueue(tokens, stream, call)


def embedding_grad(tokens: torch.Tensor, dout: torch.Tensor, n_rows: int, scale: float = 1.0,
                   out: Optional[torch.Tensor] = None, accumulate: bool = False, stream=None):
    """Gradient of ``embedding_lookup`` by the table: (n_rows, D), row v the scaled sum of dout over
    the positions that hold token v, added up in 32 bits in a fixed order.

    dout: tokens.shape + (D,).  out (n_rows, D): dout's type or float32; with ``accumulate`` the
    gradient is added to it (rows without a position keep what they hold)."""
    size = _tokens(tokens)
    _x(dout, "dout")
    if dout.dim() != tokens.dim() + 1 or dout.shape[:-1] != tokens.shape or dout.shape[-1] < 1:
        raise ValueError("dout must have shape tokens.shape + (D,)")
    _on(tokens, "dout", dout)
    if dout.dim() > 3:
        dout = dout.view(-1, dout.shape[-2], dout.shape[-1])
    stride = _rows(dout, "dout")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    n, d = tokens.numel(), dout.shape[-1]
    if not 1 <= n_rows <= 1 << 24:
        raise ValueError("n_rows must be in 1 .. 2^24")

    def call(handle):
        L = _lib()
        g = torch.empty((n_rows, d), dtype=dout.dtype, device=dout.device) if out is None else out
        _plain(g, "out", (n_rows, d), torch.float32 if g.dtype == torch.float32 else dout.dtype, dout.get_device())
        need = L.embedding_grad_workspace(n, n_rows, d)
        ws = torch.empty(need, dtype=torch.uint8, device=dout.device)
        _check(L.embedding_grad(_DTYPE[dout.dtype], _DTYPE[g.dtype], tokens.data_ptr(), size, n, dout.data_ptr(), stride,
                                n_rows, d, scale, 1 if accumulate else 0, g.data_ptr(), ws.data_ptr(), need, handle),
               "embedding_grad")
        return g

    return _enqueue(tokens, stream, call)


# ---------------------------------------------------------------------- convolution
class ConvGrads(NamedTuple):
    """Gradients of causal_conv1d; dweight and dbias are float32, dbias and dinitial_state None where the input was."""
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]
    dinitial_state: Optional[torch.Tensor]


def _conv_weights(x, weight, bias, activation):
    """(weight type code, activation code, K, D, weight address, bias address)"""
    if weight.dim() != 2:
        raise ValueError("weight must be (D, K) with K in 2 .. 4")
    d, k = weight.shape
    if d != x.shape[-1] or not 2 <= k <= 4:
        raise ValueError("weight must be (D, K) with K in 2 .. 4")
    if activation not in _ACT:
        raise ValueError("activation must be None or 'silu'")
    wt, device = weight.dtype, x.get_device()
    if wt != x.dtype and wt != torch.float32:
        raise TypeError("weight must be of x's type or float32")
    return (_DTYPE[wt], _ACT[activation], k, d, _plain(weight, "weight", (d, k), wt, device),
            _plain(bias, "bias", (d,), wt, device))


def _conv_args(x, weight, bias, activation, seq_offsets, initial_state):
    _x(x)
    rows, seqs, offsets = _lengths(x, seq_offsets)
    wt, act, k, d, w, b = _conv_weights(x, weight, bias, activation)
    state = (seqs, k - 1, d)
    a = _ConvArgs(_DTYPE[x.dtype], wt, act, k, rows, seqs, offsets, d, 0, x.data_ptr(), _rows(x, "x"), w, b,
                  _plain(initial_state, "initial_state", state, x.dtype, x.get_device()))
    return a, state


def causal_conv1d(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  activation: Optional[str] = None, seq_offsets: Optional[torch.Tensor] = None,
                  initial_state: Optional[torch.Tensor] = None, final_state=None, out: Optional[torch.Tensor] = None,
                  stream=None):
    """y[t] = act(bias + sum_k weight[:, k] * x[t - K + 1 + k]) along every sequence, per channel.

    x: (B, L, D), or (rows, D) with seq_offsets; weight (D, K), K = 2 .. 4, and bias (D,) of x's
    type or float32.  Inputs before a sequence come from initial_state (S, K - 1, D), oldest
    first, else they are zero.  final_state: a tensor (S, K - 1, D) for the last K - 1 inputs of
    every sequence, or True for a new one: (y, final_state) is returned then, else y.  Rows of y
    that belong to no sequence are not written (in a new y they hold whatever the memory held)."""
    a, state = _conv_args(x, weight, bias, activation, seq_offsets, initial_state)

    def call(handle):
        y, a.y, a.y_stride = _out(out, x, "out")
        fin, a.final_state = _optional_state(final_state, "final_state", state, x.dtype, x)
        _check(_lib().causal_conv1d(ctypes.byref(a), handle), "causal_conv1d")
        return y if fin is None else (y, fin)

    return _enqueue(x, stream, call)


def causal_conv1d_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       activation: Optional[str] = None, seq_offsets: Optional[torch.Tensor] = None,
                       initial_state: Optional[torch.Tensor] = None, dfinal_state: Optional[torch.Tensor] = None,
                       dx: Optional[torch.Tensor] = None, stream=None) -> ConvGrads:
    """Gradients of ``causal_conv1d`` (its arguments) for dy, and for dfinal_state if given.

    dx may be given to write into (a slice of a wider tensor, say); its rows that belong to no
    sequence are not written then, and are zero otherwise."""
    a, state = _conv_args(x, weight, bias, activation, seq_offsets, initial_state)
    d, k = weight.shape
    g = _ConvGradArgs(a, *_like(dy, "dy", x.shape, x.dtype, x.get_device(), x.shape[-1]),
                      _plain(dfinal_state, "dfinal_state", state, x.dtype, x.get_device()))

    def call(handle):
        L = _lib()
        ox, g.dx, g.dx_stride = _out(dx, x, "dx", _new_rows(seq_offsets))
        dw = torch.empty(d, k, dtype=torch.float32, device=x.device)
        db = None if bias is None else torch.empty(d, dtype=torch.float32, device=x.device)
        di = None if initial_state is None else torch.empty_like(initial_state)
        need = L.causal_conv1d_grad_workspace(ctypes.byref(a))
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        g.dweight, g.dbias, g.dinitial_state = dw.data_ptr(), _ptr(db), _ptr(di)
        g.workspace, g.workspace_bytes = ws.data_ptr(), need
        _check(L.causal_conv1d_grad(ctypes.byref(g), handle), "causal_conv1d_grad")
        return ConvGrads(ox, dw, db, di)

    return _enqueue(x, stream, call)


def _slots(x, slots, n_slots):
    if slots is None:
        if n_slots < x.shape[0]:
            raise ValueError("state has fewer slots than x has rows")
        return None
    return _plain(slots, "slots", (x.shape[0],), torch.int32, x.get_device())


def causal_conv1d_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                       activation: Optional[str] = None, slots: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream=None):
    """One token per row of x (rows, D): y from state[slots[i]] (its last K - 1 inputs) and x[i]; the
    state (n_slots, K - 1, D) is shifted in place.

    rows <= 65535.  slots: int32 (rows,), distinct within a call; None: row i has slot i.  A row whose slot lies
    outside the state is skipped: its row of y is not written (in a new y it holds whatever the memory held)."""
    _x(x)
    if x.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be (rows, D), state (n_slots, K - 1, D)")
    wt, act, k, d, w, b = _conv_weights(x, weight, bias, activation)
    n, device = state.shape[0], x.get_device()
    a = _ConvStepArgs(_DTYPE[x.dtype], wt, act, k, x.shape[0], n, _slots(x, slots, n), d, 0, x.data_ptr(), _rows(x, "x"), w, b,
                      _plain(state, "state", (n, k - 1, d), x.dtype, device))

    def call(handle):
        y, a.y, a.y_stride = _out(out, x, "out")
        _check(_lib().causal_conv1d_step(ctypes.byref(a), handle), "causal_conv1d_step")
        return y

    return _enqueue(x, stream, call)


# ---------------------------------------------------------------------- scan
class ScanGrads(NamedTuple):
    """Gradients of selective_scan; dA, dD, ddelta_bias and dinitial_state are float32, and None where the input was."""
    dx: torch.Tensor
    ddelta: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dD: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddelta_bias: Optional[torch.Tensor]
    dinitial_state: Optional[torch.Tensor]


def _scan_inputs(x, delta, A, B, C, D, z, delta_bias):
    """The fields of _SCAN_INPUTS."""
    if A.dim() != 2 or B.dim() < 2:
        raise ValueError("A must be (D, N), B and C x.shape[:-1] + (groups, N)")
    d, n = A.shape
    groups, shape, device, t = B.shape[-2], x.shape, x.get_device(), x.dtype
    if shape[-1] != d or not 1 <= n <= 64:
        raise ValueError("A must be (D, N) with N in 1 .. 64")
    if groups < 1 or d % groups:
        raise ValueError("the groups of B and C must divide the channels")
    bc = shape[:-1] + (groups, n)
    f32 = torch.float32
    return (d, n, groups, 0, x.data_ptr(), _rows(x, "x"), *_like(delta, "delta", shape, t, device, d),
            _plain(A, "A", (d, n), f32, device), *_like(B, "B", bc, t, device, groups * n, 2),
            *_like(C, "C", bc, t, device, groups * n, 2), _plain(D, "D", (d,), f32, device),
            *_like(z, "z", shape, t, device, d), _plain(delta_bias, "delta_bias", (d,), f32, device))


def _scan_args(x, delta, A, B, C, D, z, delta_bias, delta_softplus, seq_offsets, initial_state):
    _x(x)
    rows, seqs, offsets = _lengths(x, seq_offsets)
    inputs = _scan_inputs(x, delta, A, B, C, D, z, delta_bias)
    state = (seqs, inputs[0], inputs[1])
    return _ScanArgs(_DTYPE[x.dtype], 1 if delta_softplus else 0, rows, seqs, offsets, *inputs,
                     _plain(initial_state, "initial_state", state, torch.float32, x.get_device())), state


def selective_scan(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                   seq_offsets: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                   final_state=None, save_for_grad: bool = False, out: Optional[torch.Tensor] = None, stream=None):
    """Selective state-space scan along every sequence, per channel d (of group g) and state n:

        dt = delta + delta_bias, through softplus if delta_softplus
        h[t] = exp(dt A[d, n]) h[t-1] + dt x[t, d] B[t, g, n]
        y[t, d] = (sum_n C[t, g, n] h[t] + D[d] x[t, d]) * silu(z[t, d])

    x, delta, z: (B, L, D), or (rows, D) with seq_offsets; B, C: x.shape[:-1] + (G, N), all of x's
    type; G divides D, N <= 64.  A (D, N), D (D,), delta_bias (D,) and the states (S, D, N) are
    float32.  initial_state: h before every sequence (default zero).  final_state: a tensor for h
    after every sequence, or True for a new one.  save_for_grad: also return the states that
    ``selective_scan_grad`` starts from.  Returns y, followed by what was asked for.  Rows of y that
    belong to no sequence are not written (in a new y they hold whatever the memory held)."""
    a, state = _scan_args(x, delta, A, B, C, D, z, delta_bias, delta_softplus, seq_offsets, initial_state)

    def call(handle):
        L = _lib()
        y, a.y, a.y_stride = _out(out, x, "out")
        got = [y]
        fin, a.final_state = _optional_state(final_state, "final_state", state, torch.float32, x)
        if fin is not None:
            got.append(fin)
        if save_for_grad:
            saved = torch.empty(L.selective_scan_saved(ctypes.byref(a)), dtype=torch.float32, device=x.device)
            a.saved = saved.data_ptr()
            got.append(saved)
        need = L.selective_scan_workspace(ctypes.byref(a))
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        _check(L.selective_scan(ctypes.byref(a), handle), "selective_scan")
        return y if len(got) == 1 else tuple(got)

    return _enqueue(x, stream, call)


def selective_scan_grad(dy: torch.Tensor, x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                        seq_offsets: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                        dfinal_state: Optional[torch.Tensor] = None, saved: Optional[torch.Tensor] = None,
                        dx: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None, stream=None) -> ScanGrads:
    """Gradients of ``selective_scan`` (its arguments) for dy, and for dfinal_state if given.

    saved: what ``selective_scan(..., save_for_grad=True)`` returned for the same inputs; without
    it the states are scanned again.  dx and dz may be given to write into (two slices of one
    tensor, say).  Gradients of rows that belong to no sequence are zero, but for those of a given
    dx or dz, which are not written."""
    a, state = _scan_args(x, delta, A, B, C, D, z, delta_bias, delta_softplus, seq_offsets, initial_state)
    g = _ScanGradArgs(a, *_like(dy, "dy", x.shape, x.dtype, x.get_device(), x.shape[-1]),
                      _plain(dfinal_state, "dfinal_state", state, torch.float32, x.get_device()))
    if dz is not None and z is None:
        raise ValueError("dz given without z")

    def call(handle):
        L = _lib()
        f32 = dict(dtype=torch.float32, device=x.device)
        need_saved = L.selective_scan_saved(ctypes.byref(a))
        states = saved
        if states is None:
            states = torch.empty(need_saved, **f32)
            need = L.selective_scan_workspace(ctypes.byref(a))
            ws = torch.empty(need, dtype=torch.uint8, device=x.device)
            a.saved, a.workspace, a.workspace_bytes = states.data_ptr(), ws.data_ptr(), need
            _check(L.selective_scan(ctypes.byref(a), handle), "selective_scan")
        a.saved = _plain(states, "saved", (need_saved,), torch.float32, x.get_device())
        g.args = a
        new = _new_rows(seq_offsets)
        ox, g.dx, g.dx_stride = _out(dx, x, "dx", new)
        od, g.ddelta, g.ddelta_stride = _out(None, x, "ddelta", new)
        oz, g.dz, g.dz_stride = (None, None, 0) if z is None else _out(dz, x, "dz", new)
        oB = new(B.shape, dtype=x.dtype, device=x.device)
        oC = new(C.shape, dtype=x.dtype, device=x.device)
        oA = torch.empty(A.shape, **f32)
        oD = None if D is None else torch.empty(D.shape, **f32)
        ob = None if delta_bias is None else torch.empty(delta_bias.shape, **f32)
        oi = None if initial_state is None else torch.empty(state, **f32)
        g.dB, g.db_stride, g.dC, g.dc_stride = oB.data_ptr(), _rows(oB, "dB", 2), oC.data_ptr(), _rows(oC, "dC", 2)
        g.dA, g.dD, g.ddelta_bias, g.dinitial_state = oA.data_ptr(), _ptr(oD), _ptr(ob), _ptr(oi)
        need = L.selective_scan_grad_workspace(ctypes.byref(g))
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
        g.args.workspace, g.args.workspace_bytes = ws.data_ptr(), need
        _check(L.selective_scan_grad(ctypes.byref(g), handle), "selective_scan_grad")
        return ScanGrads(ox, od, oA, oB, oC, oD, oz, ob, oi)

    return _enqueue(x, stream, call)


def selective_scan_step(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        state: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        delta_bias: Optional[torch.Tensor] = None, delta_softplus: bool = False,
                        slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """One token per row: one step of ``selective_scan``'s recurrence from state[slots[i]], which is
    updated in place.

    x, delta, z: (rows, D); B, C: (rows, G, N); state: (n_slots, D, N) float32.  slots as in
    ``causal_conv1d_step``."""
    _x(x)
    if x.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be (rows, D), state (n_slots, D, N)")
    inputs = _scan_inputs(x, delta, A, B, C, D, z, delta_bias)
    slot_count = state.shape[0]
    a = _ScanStepArgs(_DTYPE[x.dtype], 1 if delta_softplus else 0, x.shape[0], slot_count, _slots(x, slots, slot_count), *inputs,
                      _plain(state, "state", (slot_count, inputs[0], inputs[1]), torch.float32, x.get_device()))

    def call(handle):
        y, a.y, a.y_stride = _out(out, x, "out")
        _check(_lib().selective_scan_step(ctypes.byref(a), handle), "selective_scan_step")
        return y

    return _enqueue(x, stream, call)
