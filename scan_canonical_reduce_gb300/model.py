"""Model operators of libcr: embedding lookup, layer norm, short causal
convolution, selective state space scan and gated scan, each with its gradient
and, for the last three, its form for single tokens, and sampling of the next
token (the token path of a recurrent language model).

Everything is computed in libcr's kernels (``include/cr.h``) and there is no
CPU path. The tensors are taken apart by a small native module
(``csrc/model_binding.cpp``), since a single-token call takes only a few
microseconds on the device; the functions here name its arguments. Tensors
are token-major, ``(batch, time, channel)``, of one type among float32,
bfloat16 and float16; weights, scan states and sums are float32. Tensors
whose last axis is not contiguous are copied first, as is a table or its
gradient whose rows overlap; any other strides are used as they are. ``stream``
is where the call runs (the current stream by default); copies, outputs and
the call's workspace are made on it: those of a captured call are the graph's
own.

Every result is one fixed expression of the inputs, by their shapes: repeated
calls give the same bits. (A sequence of :func:`gated_scan` may differ in its last
bits from the same one in a larger batch.)

``embedding``, ``layer_norm``, ``causal_conv``, ``selective_scan`` and
``gated_scan`` are differentiable: where autograd records, their results'
gradients are those of the ``*_backward`` calls, which may also be called
directly. Those, the single-token calls and ``sample`` are never recorded.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch
from torch.autograd.function import once_differentiable

from . import _HERE, _I32, _I64, _P, SIGNATURES, _check, lib

BINDING_PATH = os.path.join(_HERE, "_build", "cr_model_binding.so")


# The argument blocks of include/cr.h, for callers of the C ABI.
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


class _NormArgs(ctypes.Structure):
    """cr_layer_norm_args"""
    _fields_ = [("batch", _I64), ("len", _I64), ("dim", _I64), ("dt", _I32),
                ("eps", ctypes.c_float), ("x", _P), ("x_batch_stride", _I64),
                ("x_time_stride", _I64), ("weight", _P), ("bias", _P)]


class _NormGrads(ctypes.Structure):
    """cr_layer_norm_grads"""
    _fields_ = [("dy", _P), ("dy_batch_stride", _I64), ("dy_time_stride", _I64), ("stats", _P),
                ("dx", _P), ("dx_batch_stride", _I64), ("dx_time_stride", _I64),
                ("dweight", _P), ("dbias", _P)]


class _GateArgs(ctypes.Structure):
    """cr_gated_scan_args"""
    _fields_ = [("batch", _I64), ("len", _I64), ("dim", _I64), ("dt", _I32),
                ("index_bytes", _I32),
                ("x", _P), ("x_batch_stride", _I64), ("x_time_stride", _I64),
                ("gate", _P), ("gate_batch_stride", _I64), ("gate_time_stride", _I64),
                ("z", _P), ("z_batch_stride", _I64), ("z_time_stride", _I64),
                ("state", _P), ("lengths", _P)]


class _GateGrads(ctypes.Structure):
    """cr_gated_scan_grads"""
    _fields_ = [("dy", _P), ("dy_batch_stride", _I64), ("dy_time_stride", _I64), ("dfinal", _P),
                ("checkpoints", _P), ("dx", _P), ("dgate", _P), ("dz", _P), ("dstate", _P)]


class _SampleArgs(ctypes.Structure):
    """cr_sample_args"""
    _fields_ = [("rows", _I64), ("vocab", _I64), ("dt", _I32), ("index_bytes", _I32),
                ("logits", _P), ("row_stride", _I64), ("u", _P),
                ("temperature", ctypes.c_double), ("top_p", ctypes.c_double),
                ("min_p", ctypes.c_double), ("top_k", _I64), ("temperatures", _P),
                ("top_ps", _P), ("min_ps", _P), ("top_ks", _P)]


_lock = threading.Lock()


def load():
    """The native module, given the functions of the libcr that is loaded. It is
    loaded by the first call of a model operator: the reductions and scans work
    without it."""
    global _native
    with _lock:
        if isinstance(_native, _Unloaded):
            _native = _load()
    return _native


class _Unloaded:
    """Stands where the native module will be."""

    def __getattr__(self, name):
        return getattr(load(), name)


def _load():
    if not os.path.exists(BINDING_PATH):
        raise ImportError(
            "cr_model_binding.so is missing (%s): build it first with "
            "`python -c 'import __graft_entry__ as g; g.build()'`" % BINDING_PATH)
    loader = importlib.machinery.ExtensionFileLoader("cr_model_binding", BINDING_PATH)
    spec = importlib.util.spec_from_file_location("cr_model_binding", BINDING_PATH, loader=loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    names = [n for n in SIGNATURES if n.startswith((
        "cr_embedding", "cr_causal_conv", "cr_selective_scan", "cr_layer_norm", "cr_gated_scan",
        "cr_sample"))]
    module.bind({n: ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in names}, _check)
    return module


_native = _Unloaded()


# ------------------------------------------------------------- autograd
def _no_out(out) -> None:
    if out is not None:
        raise RuntimeError("a call with out= is not recorded by autograd, but one of its "
                           "arguments requires a gradient (or has a tangent)")


def _backward_on(stream, call):
    """call(stream) for a backward call, on its forward call's stream, between what
    the engine's stream has made and what it does with the results."""
    if stream is None:
        return call(None)
    here = torch.cuda.current_stream(stream.device)
    stream.wait_stream(here)
    out = call(stream)
    here.wait_stream(stream)
    for t in out.values():
        t.record_stream(here)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, stream):
        ctx.save_for_backward(tokens)
        ctx.rest = table.shape[0], table.dtype, scale, stream
        return _native.embedding(tokens, table, scale, None, stream)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (tokens,) = ctx.saved_tensors
        vocab, dtype, scale, stream = ctx.rest
        g = _backward_on(stream, lambda s: {"table": embedding_backward(tokens, dy, vocab, scale,
                                                                        stream=s)})
        return None, g["table"].to(dtype), None, None


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, state, lengths, activation, return_state, stream):
        ctx.save_for_backward(x, weight, bias, state, lengths)
        ctx.rest = activation, stream
        ctx.set_materialize_grads(False)
        return _native.causal_conv(x, weight, bias, activation, state, lengths, return_state, None,
                                   stream)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal=None):
        x, weight, bias, state, lengths = ctx.saved_tensors
        activation, stream = ctx.rest
        dy = torch.zeros_like(x) if dy is None else dy
        g = _backward_on(stream, lambda s: causal_conv_backward(
            dy, x, weight, bias, activation, state, lengths, dfinal, s))
        return g["x"], g["weight"], g.get("bias"), g.get("state"), None, None, None, None


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, dt_bias, state, lengths, softplus, return_state,
                return_checkpoints, stream):
        out = _native.selective_scan(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths,
                                     return_state, True, None, stream)
        kept = out[-1]
        ctx.mark_non_differentiable(kept)
        ctx.save_for_backward(u, dt, A, B, C, D, z, dt_bias, state, lengths, kept)
        ctx.rest = softplus, return_state, stream
        ctx.set_materialize_grads(False)
        if return_checkpoints:
            return out
        return out[:-1] if return_state else out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, *more):
        u, dt, A, B, C, D, z, dt_bias, state, lengths, kept = ctx.saved_tensors
        softplus, return_state, stream = ctx.rest
        dy = torch.zeros_like(u) if dy is None else dy
        g = _backward_on(stream, lambda s: selective_scan_backward(
            dy, u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths,
            more[0] if return_state else None, kept, s))
        return (*(g.get(k) for k in ("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "state")),
                None, None, None, None, None)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, return_stats, stream):
        y, stats = _native.layer_norm(x, weight, bias, eps, True, None, stream)
        ctx.mark_non_differentiable(stats)
        ctx.save_for_backward(x, weight, bias, stats)
        ctx.rest = eps, stream
        ctx.set_materialize_grads(False)
        return (y, stats) if return_stats else y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstats=None):
        if dy is None:
            return (None,) * 6
        x, weight, bias, stats = ctx.saved_tensors
        eps, stream = ctx.rest
        g = _backward_on(stream, lambda s: layer_norm_backward(dy, x, weight, bias, eps, stats, s))
        return g["x"], g.get("weight"), g.get("bias"), None, None, None


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, z, state, lengths, return_state, return_checkpoints, stream):
        out = _native.gated_scan(x, gate, z, state, lengths, return_state, True, None, stream)
        kept = out[-1]
        ctx.mark_non_differentiable(kept)
        ctx.save_for_backward(x, gate, z, state, lengths, kept)
        ctx.rest = return_state, stream
        ctx.set_materialize_grads(False)
        if return_checkpoints:
            return out
        return out[:-1] if return_state else out[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, *more):
        x, gate, z, state, lengths, kept = ctx.saved_tensors
        return_state, stream = ctx.rest
        dy = torch.zeros_like(x) if dy is None else dy
        g = _backward_on(stream, lambda s: gated_scan_backward(
            dy, x, gate, z, state, lengths, more[0] if return_state else None, kept, s))
        return (*(g.get(k) for k in ("x", "gate", "z", "state")), None, None, None, None)


# ------------------------------------------------------------ embedding
def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``scale * table[tokens]``: tokens (any shape, int32 or int64), table
    (vocab, dim). A token outside [0, vocab) is padding: a zero row."""
    y = _native.embedding(tokens, table, scale, out, stream)
    if y is NotImplemented:
        _no_out(out)
        return _Embedding.apply(tokens, table, scale, stream)
    return y


def embedding_backward(tokens: torch.Tensor, grad: torch.Tensor, vocab: int, scale: float = 1.0,
                       out: torch.Tensor | None = None, accumulate: bool = False,
                       stream=None) -> torch.Tensor:
    """The gradient (vocab, dim), float32, of :func:`embedding` for its table:
    row v is ``scale * tree(grad rows with token v, in order)``, tree being
    the canonical reduction's (L = 1). ``out`` receives it; with
    ``accumulate`` it is added to ``out``, whose rows without tokens stay."""
    return _native.embedding_backward(tokens, grad, vocab, scale, out, accumulate, stream)


# --------------------------------------------------------- convolution
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
    y = _native.causal_conv(x, weight, bias, activation, state, lengths, return_state, out, stream)
    if y is NotImplemented:
        _no_out(out)
        return _CausalConv.apply(x, weight, bias, state, lengths, activation, return_state, stream)
    return y


def causal_conv_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         bias: torch.Tensor | None = None, activation: str | None = None,
                         state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
                         dfinal: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`causal_conv` for the same arguments: a dict
    with "x" and "weight", and "bias" and "state" where those were given.
    ``dfinal``: the gradient of the returned state, if it was used."""
    return _native.causal_conv_backward(x, weight, bias, activation, state, lengths, dy, dfinal,
                                        stream)


def causal_conv_step(x: torch.Tensor, state: torch.Tensor, weight: torch.Tensor,
                     bias: torch.Tensor | None = None, activation: str | None = None,
                     slots: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """One token of each of ``batch`` running streams: x (batch, dim) after its
    state row, which is shifted in place. ``state`` (rows, K-1, dim),
    contiguous; stream b uses row ``slots[b]`` (b without slots); a slot
    outside [0, rows) is padding (zeros, no state changes). Slots must differ.
    Returns y (batch, dim)."""
    return _native.causal_conv_step(x, state, weight, bias, activation, slots, out, stream)


# ------------------------------------------------------ selective scan
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
    y = _native.selective_scan(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths,
                               return_state, return_checkpoints, out, stream)
    if y is NotImplemented:
        _no_out(out)
        return _SelectiveScan.apply(u, dt, A, B, C, D, z, dt_bias, state, lengths, softplus,
                                    return_state, return_checkpoints, stream)
    return y


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
    if checkpoints is None:
        with torch.no_grad():
            checkpoints = selective_scan(u, dt, A, B, C, D, None, dt_bias, softplus, state,
                                         lengths, return_checkpoints=True, stream=stream)[1]
    return _native.selective_scan_backward(u, dt, A, B, C, D, z, dt_bias, softplus, state, lengths,
                                           dy, dfinal, checkpoints, stream)


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
    return _native.selective_scan_step(u, dt, A, B, C, D, z, dt_bias, softplus, state, slots, out,
                                       stream)


# ---------------------------------------------------------- layer norm
def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5, return_stats: bool = False,
               out: torch.Tensor | None = None, stream=None):
    """``(x - mean) / sqrt(var + eps) * weight + bias`` over the last axis of x
    (any leading axes); weight and bias (dim), float32, each optional. Returns
    y, or (y, stats) with ``return_stats``: what the backward call takes of each
    row, (..., 3) float32."""
    y = _native.layer_norm(x, weight, bias, eps, return_stats, out, stream)
    if y is NotImplemented:
        _no_out(out)
        return _LayerNorm.apply(x, weight, bias, eps, return_stats, stream)
    return y


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor | None = None,
                        bias: torch.Tensor | None = None, eps: float = 1e-5,
                        stats: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`layer_norm` for the same arguments: a dict with
    "x", and "weight" and "bias" where those were given. ``stats``: from the
    forward call (computed again without them)."""
    return _native.layer_norm_backward(x, weight, bias, eps, dy, stats, stream)


# ---------------------------------------------------------- gated scan
def gated_scan(x: torch.Tensor, gate: torch.Tensor, z: torch.Tensor | None = None,
               state: torch.Tensor | None = None, lengths: torch.Tensor | None = None,
               return_state: bool = False, return_checkpoints: bool = False,
               out: torch.Tensor | None = None, stream=None):
    """Gated linear recurrence over time, per channel:

        a[t] = sigmoid(gate[t])
        h[t] = a[t] h[t-1] + (1 - a[t]) x[t]
        y[t] = h[t] * silu(z[t])

    x, gate, z (batch, time, dim), z optional; ``state`` (batch, dim), float32:
    h before time 0 (zeros without it). ``lengths`` (batch): later positions are
    not read, give zeros and leave the state. An infinite h stays infinite until it
    meets the other infinity or NaN. Returns y, followed by the last state
    (``return_state``) and the checkpoints that the backward call takes
    (``return_checkpoints``)."""
    y = _native.gated_scan(x, gate, z, state, lengths, return_state, return_checkpoints, out,
                           stream)
    if y is NotImplemented:
        _no_out(out)
        return _GatedScan.apply(x, gate, z, state, lengths, return_state, return_checkpoints,
                                stream)
    return y


def gated_scan_backward(dy: torch.Tensor, x: torch.Tensor, gate: torch.Tensor,
                        z: torch.Tensor | None = None, state: torch.Tensor | None = None,
                        lengths: torch.Tensor | None = None,
                        dfinal: torch.Tensor | None = None,
                        checkpoints: torch.Tensor | None = None, stream=None) -> dict:
    """The gradients of :func:`gated_scan` for the same arguments: a dict with
    "x" and "gate", and "z" and "state" where those were given. ``dfinal``: the
    gradient of the returned state, if it was used. ``checkpoints``: from the
    forward call (computed again without them)."""
    if checkpoints is None:
        with torch.no_grad():
            checkpoints = gated_scan(x, gate, None, state, lengths, return_checkpoints=True,
                                     stream=stream)[1]
    return _native.gated_scan_backward(x, gate, z, state, lengths, dy, dfinal, checkpoints, stream)


def gated_scan_step(x: torch.Tensor, gate: torch.Tensor, state: torch.Tensor,
                    z: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One token of each of ``batch`` running streams: x, gate, z (batch, dim).
    ``state`` (rows, dim), float32, contiguous, is updated in place; stream b
    uses row ``slots[b]`` (b without slots); a slot outside [0, rows) is padding
    (zeros, no state changes). Slots must differ. Returns y (batch, dim)."""
    return _native.gated_scan_step(x, gate, state, z, slots, out, stream)


# ------------------------------------------------------------ sampling
def sample(logits: torch.Tensor, u: torch.Tensor, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The next token of each row of logits (..., vocab), int64, from the uniform
    numbers u (...), float32 in [0, 1).

    A row's tokens, in the order of falling logits (equal ones by index), have
    the weights ``w = exp((logit - largest) / temperature)``. Kept are the first
    ``top_k`` (0: all); of these, those before which less than ``top_p`` of
    their weight lies; and of these, those with ``w >= min_p``; the first in any
    case. The token is the first whose running sum of kept weights exceeds u
    times their sum. A temperature of 0 takes the first. A logit of -inf or NaN
    is no candidate; a row without candidates gives -1, which
    :func:`embedding` takes as padding.

    Each setting is a number, or a tensor (...) with one a row: float32, and
    int32 or int64 for top_k. The result is that of exact arithmetic unless u,
    top_p or min_p lies within 2^-32 of a border (weights to 2^-32, sums in
    integers), and never differentiated."""
    return _native.sample(logits, u, temperature, top_k, top_p, min_p, out, stream)


__all__ = ["layer_norm", "layer_norm_backward", "gated_scan", "gated_scan_backward",
           "gated_scan_step", "sample", "embedding", "embedding_backward", "causal_conv",
           "causal_conv_backward", "causal_conv_step", "selective_scan",
           "selective_scan_backward", "selective_scan_step"]
