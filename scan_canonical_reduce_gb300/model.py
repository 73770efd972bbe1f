"""Model operators of libcr: embedding lookup, short causal convolution and
selective state space scan, each with its gradient and, for the last two, its
form for single tokens (the token path of a recurrent language model).

Like the rest of the binding this module only marshals tensors into the C
calls of ``include/cr.h``; everything is computed in libcr's kernels and
there is no CPU path. Tensors are token-major, ``(batch, time, channel)``, of
one type among float32, bfloat16 and float16; weights, scan states and sums
are float32. Tensors whose last axis is not contiguous are copied first; any
other strides are used as they are. ``stream`` is where the call runs (the
current stream by default); outputs are allocated on it.

Every result is one fixed expression of the inputs: repeated calls give the
same bits.
"""
from __future__ import annotations

import ctypes

import torch

from . import _P, _I32, _I64, _WS, _check, lib

_TYPES = {torch.float32: 1, torch.bfloat16: 3, torch.float16: 4}  # cr_dtype
_ACTIVATIONS = {None: 0, "silu": 1}


class _ConvArgs(ctypes.Structure):
    """cr_causal_conv_args"""
    _fields_ = [("batch", _I64), ("len", _I64), ("dim", _I64), ("width", _I32),
                ("activation", _I32), ("dt", _I32), ("index_bytes", _I32), ("x", _P),
                ("x_batch_stride", _I64), ("x_time_stride", _I64), ("weight", _P), ("bias", _P),
                ("state", _P), ("lengths", _P)]


class _ConvGrads(ctypes.Structure):
    """cr_causal_conv_grads"""
    _fields_ = [("dy", _P), ("dy_batch_stride", _I64), ("dy_time_stride", _I64), ("dfinal", _P),
                ("dx", _P), ("dx_batch_stride", _I64), ("dx_time_stride", _I64),
                ("dweight", _P), ("dbias", _P), ("dstate", _P)]


class _ScanArgs(ctypes.Structure):
    """cr_selective_scan_args"""
    _fields_ = [("batch", _I64), ("len", _I64), ("dim", _I64), ("dstate", _I32),
                ("groups", _I32), ("softplus", _I32), ("dt_type", _I32), ("index_bytes", _I32),
                ("reserved", _I32),
                ("u", _P), ("u_batch_stride", _I64), ("u_time_stride", _I64),
                ("dt", _P), ("dt_batch_stride", _I64), ("dt_time_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64), ("z_time_stride", _I64),
                ("B", _P), ("B_batch_stride", _I64), ("B_time_stride", _I64),
                ("C", _P), ("C_batch_stride", _I64), ("C_time_stride", _I64),
                ("A", _P), ("D", _P), ("dt_bias", _P), ("state", _P), ("lengths", _P)]


class _ScanGrads(ctypes.Structure):
    """cr_selective_scan_grads"""
    _fields_ = [("dy", _P), ("dy_batch_stride", _I64), ("dy_time_stride", _I64), ("dfinal", _P),
                ("checkpoints", _P), ("du", _P), ("ddt", _P), ("dz", _P), ("dB", _P), ("dC", _P),
                ("dA", _P), ("dD", _P), ("ddt_bias", _P), ("dstate", _P)]


# ------------------------------------------------------------ arguments
def _type_code(t: torch.Tensor) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("the model operators take float32, bfloat16 or float16, got %s" % t.dtype)
    return code


def _like(t, name, shape, dtype, device):
    """Checks an argument; None stays None."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    return t


def _device(t: torch.Tensor, name: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the model operators have no host form)" % name)
    return t.device


def _indices(t, name, shape, device):
    """(tensor, bytes an index) of a contiguous int32 or int64 tensor."""
    if t is None:
        return None, 4
    if t.dtype not in (torch.int32, torch.int64):
        raise TypeError("%s must be int32 or int64, got %s" % (name, t.dtype))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    return t.contiguous(), t.element_size()


def _rows(t):
    """t with a contiguous last axis (and, for B and C, last two axes)."""
    return t if t is None or t.shape[-1] <= 1 or t.stride(-1) == 1 else t.contiguous()


def _ptr(t):
    return None if t is None or t.numel() == 0 else t.data_ptr()


class _On:
    """The device and stream of a call: allocates its outputs there, and tells
    the allocator about inputs of other streams."""

    def __init__(self, device, stream):
        current = torch.cuda.current_stream(device)
        self.device = device
        self.stream = current if stream is None else stream
        self.foreign = self.stream != current
        self.ptr = self.stream.cuda_stream
        self.kept = []

    def empty(self, shape, dtype):
        if not self.foreign:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def reads(self, *tensors):
        if self.foreign:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)

    def call(self, name, *args):
        if self.device.index == torch.cuda.current_device():
            _check(getattr(lib(), name)(*args, self.ptr), name)
        else:
            with torch.cuda.device(self.device):
                _check(getattr(lib(), name)(*args, self.ptr), name)

    def workspace(self, nbytes, name):
        if nbytes == 0:
            raise ValueError("invalid %s arguments" % name)
        return _WS.get(self.device, self.stream, nbytes)


def _output(on, out, shape, dtype):
    if out is None:
        return on.empty(shape, dtype)
    _like(out, "out", shape, dtype, on.device)
    if out.shape[-1] > 1 and out.stride(-1) != 1:
        raise ValueError("out must have a contiguous last axis")
    on.reads(out)
    return out


# ------------------------------------------------------------ embedding
def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``scale * table[tokens]``: tokens (any shape, int32 or int64), table
    (vocab, dim). A token outside [0, vocab) is padding: a zero row."""
    device = _device(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be 2-D (vocab, dim)")
    dt = _type_code(table)
    tok, nbytes = _indices(tokens, "tokens", None, device)
    table = _rows(table)
    on = _On(device, stream)
    n, (vocab, dim) = tok.numel(), table.shape
    o = _output(on, out, tuple(tokens.shape) + (dim,), table.dtype)
    flat = o if o.dim() == 2 else o.view(n, dim)
    on.reads(tok, table)
    on.call("cr_embedding", _ptr(tok), nbytes, n, _ptr(table), vocab, dim,
            max(table.stride(0), dim), float(scale), dt, _ptr(flat),
            max(flat.stride(0), dim) if n > 1 else dim)
    return o


def embedding_backward(tokens: torch.Tensor, grad: torch.Tensor, vocab: int, scale: float = 1.0,
                       out: torch.Tensor | None = None, accumulate: bool = False,
                       stream=None) -> torch.Tensor:
    """The gradient (vocab, dim), float32, of :func:`embedding` for its table:
    row v is ``scale * tree(grad rows with token v, in order)``, tree being
    the canonical reduction's (L = 1). ``out`` receives it; with
    ``accumulate`` it is added to ``out``, whose rows without tokens stay."""
    device = _device(grad, "grad")
    if grad.dim() != tokens.dim() + 1 or tuple(grad.shape[:-1]) != tuple(tokens.shape):
        raise ValueError("grad must have the shape of tokens and a channel axis")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if vocab < 0:
        raise ValueError("vocab must be >= 0")
    dt = _type_code(grad)
    tok, nbytes = _indices(tokens, "tokens", None, device)
    n, dim = tok.numel(), grad.shape[-1]
    rows = _rows(grad if grad.dim() == 2 else grad.reshape(n, dim))
    if n > 1 and rows.stride(0) < dim:  # rows repeated by a zero stride
        rows = rows.contiguous()
    on = _On(device, stream)
    o = _output(on, out, (vocab, dim), torch.float32)
    ws = on.workspace(lib().cr_embedding_backward_workspace_bytes(n, vocab, dim),
                      "embedding_backward")
    on.reads(tok, rows)
    on.call("cr_embedding_backward", _ptr(tok), nbytes, n, _ptr(rows),
            rows.stride(0) if n > 1 else dim, vocab, dim, float(scale), dt, int(accumulate),
            _ptr(o), o.stride(0) if vocab > 1 else dim, ws.data_ptr(), ws.numel())
    return o


# --------------------------------------------------------- convolution
def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu', got %r" % (name,))
    return _ACTIVATIONS[name]


def _conv_args(x, weight, bias, activation, state, lengths):
    device = _device(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be (batch, time, channel)")
    dt = _type_code(x)
    batch, T, dim = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be (channel, width)")
    K = weight.shape[1]
    _like(weight, "weight", (dim, K), torch.float32, device)
    _like(bias, "bias", (dim,), torch.float32, device)
    _like(state, "state", (batch, K - 1, dim), x.dtype, device)
    lengths, ib = _indices(lengths, "lengths", (batch,), device)
    x, weight = _rows(x), weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    state = None if state is None else state.contiguous()
    a = _ConvArgs(batch, T, dim, K, _activation(activation), dt, ib, _ptr(x), x.stride(0),
                  x.stride(1), _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths))
    return device, a, (x, weight, bias, state, lengths)


def causal_conv(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
                activation: str | None = None, state: torch.Tensor | None = None,
                lengths: torch.Tensor | None = None, return_state: bool = False,
                out: torch.Tensor | None = None, stream=None):
    """Depthwise causal convolution: ``y[:, t] = act(bias + sum_k weight[:, k]
    x[:, t - (K-1) + k])``, x (batch, time, dim), weight (dim, K) with K 2 to
    4, bias (dim); weight and bias float32. ``state`` (batch, K-1, dim) holds
    the inputs before time 0 (zeros without it). ``lengths`` (batch): later
    positions are not read and give zeros. Returns y, or (y, state after the
    last position) with ``return_state``."""
    device, a, held = _conv_args(x, weight, bias, activation, state, lengths)
    on = _On(device, stream)
    y = _output(on, out, tuple(x.shape), x.dtype)
    final = on.empty((a.batch, a.width - 1, a.dim), x.dtype) if return_state else None
    on.reads(*held)
    on.call("cr_causal_conv", ctypes.byref(a), _ptr(y), y.stride(0), y.stride(1), _ptr(final))
    return (y, final) if return_state else y


def causal_conv_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         bias: torch.Tensor | None = None, activation: str | None = None,
                         state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                         dfinal: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`causal_conv` for the same arguments: a dict
    with "x" and "weight", and "bias" and "state" where those were given.
    ``dfinal``: the gradient of the returned state, if it was used."""
    device, a, held = _conv_args(x, weight, bias, activation, state, lengths)
    _like(dy, "dy", x.shape, x.dtype, device)
    _like(dfinal, "dfinal", (a.batch, a.width - 1, a.dim), x.dtype, device)
    dy = _rows(dy)
    dfinal = None if dfinal is None else dfinal.contiguous()
    on = _On(device, stream)
    g = {"x": on.empty(tuple(x.shape), x.dtype), "weight": on.empty((a.dim, a.width),
                                                                   torch.float32)}
    if bias is not None:
        g["bias"] = on.empty((a.dim,), torch.float32)
    if state is not None:
        g["state"] = on.empty((a.batch, a.width - 1, a.dim), x.dtype)
    ws = on.workspace(lib().cr_causal_conv_backward_workspace_bytes(a.batch, a.len, a.dim,
                                                                    a.width),
                      "causal_conv_backward")
    c = _ConvGrads(_ptr(dy), dy.stride(0), dy.stride(1), _ptr(dfinal), _ptr(g["x"]),
                   g["x"].stride(0), g["x"].stride(1), _ptr(g["weight"]), _ptr(g.get("bias")),
                   _ptr(g.get("state")))
    on.reads(dy, dfinal, *held)
    on.call("cr_causal_conv_backward", ctypes.byref(a), ctypes.byref(c), ws.data_ptr(),
            ws.numel())
    return g


def causal_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor,
                     bias: torch.Tensor | None = None, activation: str | None = None,
                     slots: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """One token of each of ``batch`` running streams: x (batch, dim) after its
    state row, which is shifted in place. ``state`` (rows, K-1, dim),
    contiguous; stream b uses row ``slots[b]`` (b without slots); a slot
    outside [0, rows) is padding (zeros, no state changes). Slots must differ.
    Returns y (batch, dim)."""
    device = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be (batch, dim), weight (dim, K), state (rows, K-1, dim)")
    dt = _type_code(x)
    batch, dim = x.shape
    K = weight.shape[1]
    _like(weight, "weight", (dim, K), torch.float32, device)
    _like(bias, "bias", (dim,), torch.float32, device)
    _like(state, "state", (state.shape[0], K - 1, dim), x.dtype, device)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous (it is updated in place)")
    if slots is None and state.shape[0] < batch:
        raise ValueError("state must have a row for each of the %d streams" % batch)
    slots, ib = _indices(slots, "slots", (batch,), device)
    x, weight = _rows(x), weight.contiguous()
    bias = None if bias is None else bias.contiguous()
    on = _On(device, stream)
    y = _output(on, out, (batch, dim), x.dtype)
    on.reads(x, state, weight, bias, slots)
    on.call("cr_causal_conv_step", _ptr(x), x.stride(0), _ptr(state), state.shape[0],
            _ptr(slots), ib, _ptr(weight), _ptr(bias), _activation(activation), batch, dim, K,
            dt, _ptr(y), y.stride(0))
    return y


# ------------------------------------------------------ selective scan
def _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, step):
    device = _device(u, "u")
    lead = 1 if step else 2
    if u.dim() != lead + 1:
        raise ValueError("u must be (batch, dim)" if step else "u must be (batch, time, dim)")
    code = _type_code(u)
    batch, dim = u.shape[0], u.shape[-1]
    T = 1 if step else u.shape[1]
    if A.dim() != 2:
        raise ValueError("A must be (dim, dstate)")
    N = A.shape[1]
    if B.dim() == lead + 1:  # one group
        B = B.unsqueeze(lead)
    if C.dim() == lead + 1:
        C = C.unsqueeze(lead)
    groups = B.shape[lead] if B.dim() == lead + 2 else 0
    if groups < 1 or dim % groups:
        raise ValueError("B must be (..., groups, dstate) with groups dividing dim")
    _like(dt, "dt", u.shape, u.dtype, device)
    _like(z, "z", u.shape, u.dtype, device)
    _like(B, "B", tuple(u.shape[:-1]) + (groups, N), u.dtype, device)
    _like(C, "C", tuple(u.shape[:-1]) + (groups, N), u.dtype, device)
    _like(A, "A", (dim, N), torch.float32, device)
    _like(D, "D", (dim,), torch.float32, device)
    _like(dt_bias, "dt_bias", (dim,), torch.float32, device)
    u, dt, z = _rows(u), _rows(dt), _rows(z)
    if N > 1 and (B.stride(-1) != 1 or (groups > 1 and B.stride(-2) != N)):
        B = B.contiguous()
    if N > 1 and (C.stride(-1) != 1 or (groups > 1 and C.stride(-2) != N)):
        C = C.contiguous()
    if N == 1 and groups > 1:
        B, C = B.contiguous(), C.contiguous()
    A = A.contiguous()
    D = None if D is None else D.contiguous()
    dt_bias = None if dt_bias is None else dt_bias.contiguous()
    if not step:
        _like(state, "state", (batch, dim, N), torch.float32, device)
        state = None if state is None else state.contiguous()
    lengths, ib = _indices(lengths, "slots" if step else "lengths", (batch,), device)
    t = 0 if step else 1

    def strides(v):
        return (None, 0, 0) if v is None else (_ptr(v), v.stride(0), v.stride(t) if t else 0)

    a = _ScanArgs(batch, T, dim, N, groups, int(bool(softplus)), code, ib, 0, *strides(u),
                  *strides(dt), *strides(z), *strides(B), *strides(C), _ptr(A), _ptr(D),
                  _ptr(dt_bias), None if step else _ptr(state), None if step else _ptr(lengths))
    return device, a, (u, dt, z, B, C, A, D, dt_bias, state, lengths)


def selective_scan(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                   C: torch.Tensor, D: torch.Tensor | None = None,
                   z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
                   softplus: bool = True, state: torch.Tensor | None = None,
                   lengths: torch.Tensor | None = None, return_state: bool = False,
                   return_checkpoints: bool = False, out: torch.Tensor | None = None,
                   stream=None):
    """Selective state space scan over time, per channel d and state n:

        delta = softplus(dt + dt_bias)
        h[t] = exp(delta[t] A) h[t-1] + delta[t] u[t] B[t]
        y[t] = (sum_n C[t] h[t] + D u[t]) * silu(z[t])

    u, dt, z (batch, time, dim); B, C (batch, time, groups, dstate) or
    (batch, time, dstate), a group serving dim / groups consecutive channels;
    A (dim, dstate), D, dt_bias (dim), state (batch, dim, dstate), float32.
    D, z, dt_bias and state are optional, ``softplus=False`` takes dt +
    dt_bias as it is. ``lengths`` (batch): later positions are not read, give
    zeros and leave the state. Returns y, followed by the last state
    (``return_state``) and the checkpoints that the backward call takes
    (``return_checkpoints``)."""
    device, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, False)
    on = _On(device, stream)
    y = _output(on, out, tuple(u.shape), u.dtype)
    final = on.empty((a.batch, a.dim, a.dstate), torch.float32) if return_state else None
    kept = None
    if return_checkpoints:
        kept = on.empty((a.batch, lib().cr_selective_scan_checkpoints(a.len), a.dim, a.dstate),
                        torch.float32)
    ws = on.workspace(lib().cr_selective_scan_workspace_bytes(a.batch, a.len, a.dim, a.dstate),
                      "selective_scan")
    on.reads(*held)
    on.call("cr_selective_scan", ctypes.byref(a), _ptr(y), y.stride(0), y.stride(1), _ptr(final),
            _ptr(kept), ws.data_ptr(), ws.numel())
    result = (y,) + ((final,) if return_state else ()) + ((kept,) if return_checkpoints else ())
    return result if len(result) > 1 else y


def selective_scan_backward(dy: torch.Tensor, u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                            B: torch.Tensor, C: torch.Tensor, D: torch.Tensor | None = None,
                            z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
                            softplus: bool = True, state: torch.Tensor | None = None,
                            lengths: torch.Tensor | None = None,
                            dfinal: torch.Tensor | None = None,
                            checkpoints: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`selective_scan` for the same arguments: a dict
    with "u", "dt", "A", "B", "C", and "D", "z", "dt_bias", "state" where
    those were given. ``dfinal``: the gradient of the returned state, if it
    was used. ``checkpoints``: from the forward call (computed again without
    them)."""
    device, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, False)
    _like(dy, "dy", u.shape, u.dtype, device)
    _like(dfinal, "dfinal", (a.batch, a.dim, a.dstate), torch.float32, device)
    n_check = lib().cr_selective_scan_checkpoints(a.len)
    if checkpoints is None:
        checkpoints = selective_scan(u, dt, A, B, C, D, None, dt_bias, softplus, state, lengths,
                                     return_checkpoints=True, stream=stream)[1]
    _like(checkpoints, "checkpoints", (a.batch, n_check, a.dim, a.dstate), torch.float32, device)
    if not checkpoints.is_contiguous():
        raise ValueError("checkpoints must be contiguous, as the forward call returns them")
    dy = _rows(dy)
    dfinal = None if dfinal is None else dfinal.contiguous()
    on = _On(device, stream)
    f32 = torch.float32
    g = {"u": on.empty(tuple(u.shape), u.dtype), "dt": on.empty(tuple(u.shape), u.dtype),
         "A": on.empty((a.dim, a.dstate), f32), "B": on.empty(tuple(B.shape), u.dtype),
         "C": on.empty(tuple(C.shape), u.dtype)}
    if D is not None:
        g["D"] = on.empty((a.dim,), f32)
    if z is not None:
        g["z"] = on.empty(tuple(u.shape), u.dtype)
    if dt_bias is not None:
        g["dt_bias"] = on.empty((a.dim,), f32)
    if state is not None:
        g["state"] = on.empty((a.batch, a.dim, a.dstate), f32)
    ws = on.workspace(lib().cr_selective_scan_backward_workspace_bytes(
        a.batch, a.len, a.dim, a.dstate, a.groups), "selective_scan_backward")
    c = _ScanGrads(_ptr(dy), dy.stride(0), dy.stride(1), _ptr(dfinal), _ptr(checkpoints),
                   *(_ptr(g.get(k)) for k in ("u", "dt", "z", "B", "C", "A", "D", "dt_bias",
                                              "state")))
    on.reads(dy, dfinal, checkpoints, *held)
    on.call("cr_selective_scan_backward", ctypes.byref(a), ctypes.byref(c), ws.data_ptr(),
            ws.numel())
    return g


def selective_scan_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        C: torch.Tensor, state: torch.Tensor, D: torch.Tensor | None = None,
                        z: torch.Tensor | None = None, dt_bias: torch.Tensor | None = None,
                        softplus: bool = True, slots: torch.Tensor | None = None,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of each of ``batch`` running streams: u, dt, z (batch, dim),
    B, C (batch, groups, dstate) or (batch, dstate). ``state`` (rows, dim,
    dstate), float32, contiguous, is updated in place; stream b uses row
    ``slots[b]`` (b without slots); a slot outside [0, rows) is padding
    (zeros, no state changes). Slots must differ. Returns y (batch, dim)."""
    device, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, None, slots, True)
    if state.dim() != 3:
        raise ValueError("state must be (rows, dim, dstate)")
    _like(state, "state", (state.shape[0], a.dim, a.dstate), torch.float32, device)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous (it is updated in place)")
    if slots is None and state.shape[0] < a.batch:
        raise ValueError("state must have a row for each of the %d streams" % a.batch)
    on = _On(device, stream)
    y = _output(on, out, (a.batch, a.dim), u.dtype)
    on.reads(state, *held)
    on.call("cr_selective_scan_step", ctypes.byref(a), _ptr(state), state.shape[0],
            _ptr(held[-1]), _ptr(y), y.stride(0))
    return y


__all__ = ["embedding", "embedding_backward", "causal_conv", "causal_conv_backward",
           "causal_conv_step", "selective_scan", "selective_scan_backward",
           "selective_scan_step"]
