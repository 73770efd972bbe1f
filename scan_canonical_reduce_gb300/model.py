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
import functools
import struct

import torch

from . import _P, _I32, _I64, _WS, _check, lib

_TYPES = {torch.float32: 1, torch.bfloat16: 3, torch.float16: 4}  # cr_dtype
_ACTIVATIONS = {None: 0, "silu": 1}
_F32 = torch.float32

# A single-token call is a few microseconds on the device, so the host side is
# kept to what it must do: one test an argument, no temporary objects, and the
# argument blocks packed at once.
_current_stream = torch._C._cuda_getCurrentRawStream  # of a device index, as an integer
_current_device = torch._C._cuda_getDevice


def _entry(name):
    """A libcr function that raises on an error code."""
    fn = getattr(lib(), name)

    def call(*args):
        code = fn(*args)
        if code:
            _check(code, name)
    return call


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


def _packer(structure):
    """struct.Struct with the layout of a ctypes Structure."""
    codes = {_I64: "q", _I32: "i", _P: "P"}
    packed = struct.Struct("@" + "".join(codes[t] for _, t in structure._fields_))
    assert packed.size == ctypes.sizeof(structure)
    return packed.pack


_pack_conv, _pack_conv_grads = _packer(_ConvArgs), _packer(_ConvGrads)
_pack_scan, _pack_scan_grads = _packer(_ScanArgs), _packer(_ScanGrads)

_c_embedding = _entry("cr_embedding")
_c_embedding_backward = _entry("cr_embedding_backward")
_c_conv = _entry("cr_causal_conv")
_c_conv_backward = _entry("cr_causal_conv_backward")
_c_conv_step = _entry("cr_causal_conv_step")
_c_scan = _entry("cr_selective_scan")
_c_scan_backward = _entry("cr_selective_scan_backward")
_c_scan_step = _entry("cr_selective_scan_step")


# workspace sizes and checkpoint counts of the shapes a program keeps using
@functools.lru_cache(maxsize=256)
def _size(name, *sizes):
    return getattr(lib(), name)(*sizes)


# ------------------------------------------------------------ arguments
def _type_code(t: torch.Tensor) -> int:
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError("the model operators take float32, bfloat16 or float16, got %s" % t.dtype)
    return code


def _need(t, name, shape, dtype, index):
    """Raises unless t has this shape and type and is on CUDA device `index`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index:
        return
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))


def _device(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (the model operators have no host form)" % name)
    return t.get_device()


def _indices(t, name, shape, index):
    """A contiguous int32 or int64 tensor (None stays None)."""
    if t is None:
        return None
    if t.dtype is not torch.int32 and t.dtype is not torch.int64:
        raise TypeError("%s must be int32 or int64, got %s" % (name, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if t.get_device() != index:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, index, t.device))
    return t if t.is_contiguous() else t.contiguous()


def _rows(t):
    """t with a contiguous last axis."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def _dense(t):
    return t if t.is_contiguous() else t.contiguous()


class _On:
    """Where a call runs: its device index, its stream, the stream's handle.
    With a stream other than the current one, outputs are allocated on it and
    the allocator is told which inputs it reads."""
    __slots__ = ("index", "stream", "ptr")

    def __init__(self, index, stream):
        self.index = index
        self.stream = None
        self.ptr = _current_stream(index)
        if stream is not None and stream.cuda_stream != self.ptr:
            self.stream = stream
            self.ptr = stream.cuda_stream

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.index)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.index)

    def like(self, t):
        """An uninitialised contiguous tensor of t's shape and type."""
        if self.stream is None and t.is_contiguous():
            return torch.empty_like(t)
        return self.empty(t.shape, t.dtype)

    def output(self, out, shape, dtype):
        if out is None:
            return self.empty(shape, dtype)
        _need(out, "out", shape, dtype, self.index)
        if out.stride(-1) != 1 and out.shape[-1] > 1:
            raise ValueError("out must have a contiguous last axis")
        return out

    def run(self, call, tensors, *args):
        """call(*args, stream), which uses `tensors`."""
        if self.stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(self.stream)
        if self.index == _current_device():
            call(*args, self.ptr)
        else:
            with torch.cuda.device(self.index):
                call(*args, self.ptr)

    def workspace(self, nbytes, name):
        if nbytes == 0:
            raise ValueError("invalid %s arguments" % name)
        buf = _WS._bufs.get((self.index, self.ptr))
        if buf is None or buf.numel() < nbytes:
            where = torch.device("cuda", self.index)
            buf = _WS.get(where, self.stream or torch.cuda.current_stream(where), nbytes)
        return buf


# ------------------------------------------------------------ embedding
def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``scale * table[tokens]``: tokens (any shape, int32 or int64), table
    (vocab, dim). A token outside [0, vocab) is padding: a zero row."""
    index = _device(table, "table")
    if table.dim() != 2:
        raise ValueError("table must be 2-D (vocab, dim)")
    code = _type_code(table)
    tok = _indices(tokens, "tokens", None, index)
    table = _rows(table)
    on = _On(index, stream)
    n, (vocab, dim) = tok.numel(), table.shape
    o = on.output(out, tokens.shape + (dim,), table.dtype)
    flat = o if o.dim() == 2 else o.view(n, dim)
    on.run(_c_embedding, (tok, table, o), tok.data_ptr(), tok.element_size(), n, table.data_ptr(),
           vocab, dim, max(table.stride(0), dim), scale, code, flat.data_ptr(),
           max(flat.stride(0), dim))
    return o


def embedding_backward(tokens: torch.Tensor, grad: torch.Tensor, vocab: int, scale: float = 1.0,
                       out: torch.Tensor | None = None, accumulate: bool = False,
                       stream=None) -> torch.Tensor:
    """The gradient (vocab, dim), float32, of :func:`embedding` for its table:
    row v is ``scale * tree(grad rows with token v, in order)``, tree being
    the canonical reduction's (L = 1). ``out`` receives it; with
    ``accumulate`` it is added to ``out``, whose rows without tokens stay."""
    index = _device(grad, "grad")
    if grad.dim() != tokens.dim() + 1 or grad.shape[:-1] != tokens.shape:
        raise ValueError("grad must have the shape of tokens and a channel axis")
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if vocab < 0:
        raise ValueError("vocab must be >= 0")
    code = _type_code(grad)
    tok = _indices(tokens, "tokens", None, index)
    n, dim = tok.numel(), grad.shape[-1]
    rows = _rows(grad if grad.dim() == 2 else grad.reshape(n, dim))
    if n > 1 and rows.stride(0) < dim:  # rows repeated by a zero stride
        rows = rows.contiguous()
    on = _On(index, stream)
    o = on.output(out, (vocab, dim), _F32)
    ws = on.workspace(_size("cr_embedding_backward_workspace_bytes", n, vocab, dim),
                      "embedding_backward")
    on.run(_c_embedding_backward, (tok, rows, o), tok.data_ptr(), tok.element_size(), n,
           rows.data_ptr(), rows.stride(0) if n > 1 else dim, vocab, dim, scale, code,
           int(accumulate), o.data_ptr(), o.stride(0) if vocab > 1 else dim, ws.data_ptr(),
           ws.numel())
    return o


# --------------------------------------------------------- convolution
def _activation(name) -> int:
    if name not in _ACTIVATIONS:
        raise ValueError("activation must be None or 'silu', got %r" % (name,))
    return _ACTIVATIONS[name]


def _conv_args(x, weight, bias, activation, state, lengths):
    index = _device(x, "x")
    if x.dim() != 3:
        raise ValueError("x must be (batch, time, channel)")
    code = _type_code(x)
    batch, T, dim = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be (channel, width)")
    K = weight.shape[1]
    _need(weight, "weight", (dim, K), _F32, index)
    x, weight = _rows(x), _dense(weight)
    b = st = ln = 0
    if bias is not None:
        _need(bias, "bias", (dim,), _F32, index)
        bias = _dense(bias)
        b = bias.data_ptr()
    if state is not None:
        _need(state, "state", (batch, K - 1, dim), x.dtype, index)
        state = _dense(state)
        st = state.data_ptr()
    ib = 4
    if lengths is not None:
        lengths = _indices(lengths, "lengths", (batch,), index)
        ln, ib = lengths.data_ptr(), lengths.element_size()
    xs = x.stride()
    a = _pack_conv(batch, T, dim, K, _activation(activation), code, ib, x.data_ptr(), xs[0], xs[1],
                   weight.data_ptr(), b, st, ln)
    return index, a, (x, weight, bias, state, lengths)


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
    index, a, held = _conv_args(x, weight, bias, activation, state, lengths)
    on = _On(index, stream)
    y = on.like(x) if out is None else on.output(out, x.shape, x.dtype)
    final = None
    if return_state:
        final = on.empty((x.shape[0], weight.shape[1] - 1, x.shape[2]), x.dtype)
    ys = y.stride()
    on.run(_c_conv, held + (y,), a, y.data_ptr(), ys[0], ys[1],
           final.data_ptr() if return_state else None)
    return (y, final) if return_state else y


def causal_conv_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         bias: torch.Tensor | None = None, activation: str | None = None,
                         state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                         dfinal: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`causal_conv` for the same arguments: a dict
    with "x" and "weight", and "bias" and "state" where those were given.
    ``dfinal``: the gradient of the returned state, if it was used."""
    index, a, held = _conv_args(x, weight, bias, activation, state, lengths)
    (batch, T, dim), K = x.shape, weight.shape[1]
    _need(dy, "dy", x.shape, x.dtype, index)
    dy = _rows(dy)
    if dfinal is not None:
        _need(dfinal, "dfinal", (batch, K - 1, dim), x.dtype, index)
        dfinal = _dense(dfinal)
    on = _On(index, stream)
    g = {"x": on.like(x), "weight": on.like(weight)}
    db = ds = 0
    if bias is not None:
        g["bias"] = on.like(bias)
        db = g["bias"].data_ptr()
    if state is not None:
        g["state"] = on.like(state)
        ds = g["state"].data_ptr()
    ws = on.workspace(_size("cr_causal_conv_backward_workspace_bytes", batch, T, dim, K),
                      "causal_conv_backward")
    ys, xs = dy.stride(), g["x"].stride()
    c = _pack_conv_grads(dy.data_ptr(), ys[0], ys[1], 0 if dfinal is None else dfinal.data_ptr(),
                         g["x"].data_ptr(), xs[0], xs[1], g["weight"].data_ptr(), db, ds)
    on.run(_c_conv_backward, held + (dy, dfinal), a, c, ws.data_ptr(), ws.numel())
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
    index = _device(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or state.dim() != 3:
        raise ValueError("x must be (batch, dim), weight (dim, K), state (rows, K-1, dim)")
    code = _type_code(x)
    batch, dim = x.shape
    K, rows = weight.shape[1], state.shape[0]
    _need(weight, "weight", (dim, K), _F32, index)
    _need(state, "state", (rows, K - 1, dim), x.dtype, index)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous (it is updated in place)")
    x, weight = _rows(x), _dense(weight)
    b = sl = 0
    ib = 4
    if bias is not None:
        _need(bias, "bias", (dim,), _F32, index)
        bias = _dense(bias)
        b = bias.data_ptr()
    if slots is not None:
        slots = _indices(slots, "slots", (batch,), index)
        sl, ib = slots.data_ptr(), slots.element_size()
    elif rows < batch:
        raise ValueError("state must have a row for each of the %d streams" % batch)
    on = _On(index, stream)
    y = on.like(x) if out is None else on.output(out, x.shape, x.dtype)
    on.run(_c_conv_step, (x, state, weight, bias, slots, y), x.data_ptr(), x.stride(0),
           state.data_ptr(), rows, sl, ib, weight.data_ptr(), b, _activation(activation), batch,
           dim, K, code, y.data_ptr(), y.stride(0))
    return y


# ------------------------------------------------------ selective scan
def _states(t, name, lead, N, dtype, index):
    """B or C as (..., groups, N) with the last two axes contiguous."""
    if t.dim() == len(lead) + 1:  # one group
        t = t.unsqueeze(-2)
    _need(t, name, lead + (t.shape[-2], N), dtype, index)
    s = t.stride()
    if (N > 1 and s[-1] != 1) or (t.shape[-2] > 1 and s[-2] != N):
        t = t.contiguous()
    return t


def _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, step):
    """(device index, packed argument block, tensors that it points to)."""
    index = _device(u, "u")
    shape, dtype = u.shape, u.dtype
    if len(shape) != (2 if step else 3):
        raise ValueError("u must be (batch, dim)" if step else "u must be (batch, time, dim)")
    code = _type_code(u)
    batch, dim = shape[0], shape[-1]
    if A.dim() != 2:
        raise ValueError("A must be (dim, dstate)")
    N = A.shape[1]
    _need(A, "A", (dim, N), _F32, index)
    _need(dt, "dt", shape, dtype, index)
    B = _states(B, "B", shape[:-1], N, dtype, index)
    C = _states(C, "C", shape[:-1], N, dtype, index)
    groups = B.shape[-2]
    if groups < 1 or dim % groups or C.shape[-2] != groups:
        raise ValueError("B and C must be (..., groups, dstate) with groups dividing dim")
    u, dt, A = _rows(u), _rows(dt), _dense(A)
    us, ds, bs, cs = u.stride(), dt.stride(), B.stride(), C.stride()
    zs = (0, 0)
    zp = Dp = bp = sp = lp = 0
    if z is not None:
        _need(z, "z", shape, dtype, index)
        z = _rows(z)
        zs, zp = z.stride(), z.data_ptr()
    if D is not None:
        _need(D, "D", (dim,), _F32, index)
        D = _dense(D)
        Dp = D.data_ptr()
    if dt_bias is not None:
        _need(dt_bias, "dt_bias", (dim,), _F32, index)
        dt_bias = _dense(dt_bias)
        bp = dt_bias.data_ptr()
    if state is not None:
        _need(state, "state", (batch, dim, N), _F32, index)
        state = _dense(state)
        sp = state.data_ptr()
    ib = 4
    if lengths is not None:  # of a step: its slots
        lengths = _indices(lengths, "slots" if step else "lengths", (batch,), index)
        ib = lengths.element_size()
        lp = 0 if step else lengths.data_ptr()
    a = _pack_scan(batch, 1 if step else shape[1], dim, N, groups, 1 if softplus else 0, code, ib,
                   0, u.data_ptr(), us[0], us[1], dt.data_ptr(), ds[0], ds[1], zp, zs[0], zs[1],
                   B.data_ptr(), bs[0], bs[1], C.data_ptr(), cs[0], cs[1], A.data_ptr(), Dp, bp,
                   sp, lp)
    return index, a, (u, dt, z, B, C, A, D, dt_bias, state, lengths)


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
    index, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, False)
    (batch, T, dim), N = u.shape, A.shape[1]
    on = _On(index, stream)
    y = on.like(u) if out is None else on.output(out, u.shape, u.dtype)
    final = kept = None
    if return_state:
        final = on.empty((batch, dim, N), _F32)
    if return_checkpoints:
        kept = on.empty((batch, _size("cr_selective_scan_checkpoints", T), dim, N), _F32)
    ws = on.workspace(_size("cr_selective_scan_workspace_bytes", batch, T, dim, N),
                      "selective_scan")
    ys = y.stride()
    on.run(_c_scan, held + (y,), a, y.data_ptr(), ys[0], ys[1],
           final.data_ptr() if return_state else None,
           kept.data_ptr() if return_checkpoints else None, ws.data_ptr(), ws.numel())
    if return_state:
        return (y, final, kept) if return_checkpoints else (y, final)
    return (y, kept) if return_checkpoints else y


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
    index, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths, False)
    (batch, T, dim), N, groups = u.shape, A.shape[1], held[3].shape[-2]
    _need(dy, "dy", u.shape, u.dtype, index)
    dy = _rows(dy)
    if dfinal is not None:
        _need(dfinal, "dfinal", (batch, dim, N), _F32, index)
        dfinal = _dense(dfinal)
    if checkpoints is None:
        checkpoints = selective_scan(u, dt, A, B, C, D, None, dt_bias, softplus, state, lengths,
                                     return_checkpoints=True, stream=stream)[1]
    _need(checkpoints, "checkpoints",
          (batch, _size("cr_selective_scan_checkpoints", T), dim, N), _F32, index)
    if not checkpoints.is_contiguous():
        raise ValueError("checkpoints must be contiguous, as the forward call returns them")
    on = _On(index, stream)
    g = {"u": on.like(u), "dt": on.like(dt), "A": on.like(A), "B": on.like(B), "C": on.like(C)}
    for name, t in (("D", D), ("z", z), ("dt_bias", dt_bias), ("state", state)):
        if t is not None:
            g[name] = on.like(t)
    ws = on.workspace(_size("cr_selective_scan_backward_workspace_bytes", batch, T, dim, N, groups),
                      "selective_scan_backward")
    ys = dy.stride()
    c = _pack_scan_grads(dy.data_ptr(), ys[0], ys[1], 0 if dfinal is None else dfinal.data_ptr(),
                         checkpoints.data_ptr(),
                         *(g[k].data_ptr() if k in g else 0
                           for k in ("u", "dt", "z", "B", "C", "A", "D", "dt_bias", "state")))
    on.run(_c_scan_backward, held + (dy, dfinal, checkpoints), a, c, ws.data_ptr(), ws.numel())
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
    index, a, held = _scan_args(u, dt, A, B, C, D, z, dt_bias, softplus, None, slots, True)
    batch, dim = u.shape
    if state.dim() != 3:
        raise ValueError("state must be (rows, dim, dstate)")
    rows = state.shape[0]
    _need(state, "state", (rows, dim, A.shape[1]), _F32, index)
    if not state.is_contiguous():
        raise ValueError("state must be contiguous (it is updated in place)")
    if slots is None and rows < batch:
        raise ValueError("state must have a row for each of the %d streams" % batch)
    on = _On(index, stream)
    y = on.like(u) if out is None else on.output(out, u.shape, u.dtype)
    on.run(_c_scan_step, held + (state, y), a, state.data_ptr(), rows,
           None if slots is None else held[-1].data_ptr(), y.data_ptr(), y.stride(0))
    return y


__all__ = ["embedding", "embedding_backward", "causal_conv", "causal_conv_backward",
           "causal_conv_step", "selective_scan", "selective_scan_backward",
           "selective_scan_step"]
