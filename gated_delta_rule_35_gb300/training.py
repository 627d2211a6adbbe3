"""What training a recurrent mixing layer takes beside its forward operators: the gated
linear recurrence (``recur_fwd``, ``recur_step``) with its backward pass (``recur_bwd``),
layer norm (``layer_norm``) with its own (``layer_norm_bwd``), and the short convolution's
(``conv_bwd``).

The conventions are those of the mixer operators: arguments are marshalled only, the work
runs on the current stream of the tensors' device (or on ``stream``), and the contracts are
those of include/gdn.h. Inputs marked *strided* may be slices of wider tensors. ``lengths``
([B] int32, on the device) holds the valid tokens of each sequence of a padded batch: rows
at or past it are not used, add nothing to a gradient, and are not written in the outputs
(zeros, then, in an output that the call allocates). A backward pass returns gradients; it
adds to nothing. Autograd records none of these calls: outputs do not require gradients. A
buffer for a gradient that the call does not have (of a weight, bias, gate, rate or state
that is not given) is refused; one whose output_* flag is off is left alone.
"""
from __future__ import annotations

import ctypes

import torch

from .mixer import (_INVALID, _act, _call, _dense, _form, _int32, _keep, _new, _on_stream, _plans, _ptr, _tokens,
                    _x)
from .native import DTYPES, GDN_ERR_UNSUPPORTED, GdnError, _workspace, lib

SCALINGS = {"none": 0, "complement": 1, "root": 2}
GDN_LAYER_NORM_RMS = 1
RECUR_EVERY = 16     # tokens from one kept state to the next


class RecurProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "dtype", "scaling", "reserved")] + \
               [(f"{n}_stride_{a}", ctypes.c_int64) for n in ("x", "decay", "gate", "dy") for a in "bt"]


class LayerNormProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "dtype", "flags")] + \
               [("eps", ctypes.c_float)] + [(f"{n}_stride_{a}", ctypes.c_int64) for n in ("x", "dy") for a in "bt"]


class ConvBwdProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "W", "dtype", "act")] + \
               [(f"{n}_stride_{a}", ctypes.c_int64) for n in ("x", "dy") for a in "bt"]


def _need(name, p, refusal):
    """A problem's workspace bytes, or its refusal."""
    need = getattr(lib(), name)(ctypes.byref(p))
    if need == _INVALID:
        raise GdnError(refusal(p), name)
    return need


def _scaling(scaling):
    s = SCALINGS.get(scaling)
    if s is None:
        raise ValueError(f"scaling must be one of {', '.join(SCALINGS)}")
    return s


def _optional(t, name, shape, dtype, index):
    return (0, 0) if t is None else _tokens(t, name, shape, dtype, index)


def _given(**tensors):
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} must be given")


def _zeros(shape, dtype, x, lengths=None):
    return (torch.empty if lengths is None else torch.zeros)(shape, dtype=dtype, device=x.device)


# -------------------------------------------------------- gated linear recurrence
def _recur_refusal(p):
    return lib().gdn_recur_fwd(ctypes.byref(p), *[None] * 10)


def _recur_problem(x, decay, rate, gate, scaling, lengths, dy=None):
    """(problem, device index) of the inputs that both passes take."""
    _given(decay=decay)
    shape, dtype, index = _x(x, "[B,T,D]")
    B, T, D = shape
    p = RecurProblem(*_int32("gdn_recur_fwd", B, T, D), DTYPES[dtype], _scaling(scaling), 0,
                     *_tokens(x, "x", shape, dtype, index), *_tokens(decay, "decay", shape, dtype, index),
                     *_optional(gate, "gate", shape, dtype, index), *_optional(dy, "dy", shape, dtype, index))
    _dense(rate, "rate", (D,), torch.float32, index)
    _dense(lengths, "lengths", (B,), torch.int32, index)
    return p, index


def _recur_states(x):
    B, T, D = x.shape
    return (B, (T + RECUR_EVERY - 1) // RECUR_EVERY, D)


def _recur_plan(x, decay, rate, gate, scaling, h0, lengths, out, final_state, states):
    p, index = _recur_problem(x, decay, rate, gate, scaling, lengths)
    state, kept = (x.shape[0], x.shape[2]), _recur_states(x)
    for t, name, form, kind in ((h0, "h0", state, torch.float32), (out, "out", x.shape, x.dtype),
                                (final_state, "final_state", state, torch.float32),
                                (states, "states", kept, torch.float32)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), state, kept, index


@_on_stream
def recur_fwd(x, decay, rate=None, gate=None, scaling: str = "root", h0=None, lengths=None,
              output_final_state: bool = True, output_states: bool = False, out=None, final_state=None,
              states=None):
    """Gated linear recurrence (gdn_recur_fwd). Returns (y, h_final or None), or with
    ``output_states`` (y, h_final or None, states):

        s = sigmoid(decay);  a = exp(-rate s)            (a = s without a rate)
        h <- a h + m sigmoid(gate) x,  y = h             (m x without a gate)

    per token and channel, m by ``scaling``: "root" sqrt(1 - a^2), "complement" 1 - a,
    "none" 1. x, decay, gate [B,T,D] float32 or bfloat16 (one dtype), strided; rate [D] in
    0..2^64, h0 and h_final [B,D] float32. ``states`` [B, ceil(T / RECUR_EVERY), D] float32: the
    ones entering every RECUR_EVERY-th token, for recur_bwd. ``final_state=h0`` updates the
    state in place; ``out`` and ``states`` may be passed to reuse buffers."""
    if not output_states:
        states = None
    key = ("recur", x.shape, x.stride(), x.dtype, x.get_device(), _form(decay), _form(rate), _form(gate), scaling,
           _form(h0), _form(lengths), _form(out), _form(final_state), _form(states))
    p, state, kept, index = _plans.get(key) or _keep(key, _recur_plan(
        x, decay, rate, gate, scaling, h0, lengths, out, final_state, states))
    if out is None:
        out = _new(x, lengths)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty(state, dtype=torch.float32, device=x.device)
    if output_states and states is None:
        states = _zeros(kept, torch.float32, x, lengths)
    _call(lib().gdn_recur_fwd, "gdn_recur_fwd", index, p, x.data_ptr(), decay.data_ptr(), _ptr(gate), _ptr(rate),
          _ptr(h0), _ptr(lengths), out.data_ptr(), _ptr(final_state), _ptr(states))
    return (out, final_state, states) if output_states else (out, final_state)


@_on_stream
def recur_step(x, decay, state, rate=None, gate=None, scaling: str = "root", state_out=None, out=None):
    """recur_fwd for the next token(s) of every sequence: advances ``state`` [B,D] float32
    by x's T tokens, in place unless ``state_out`` is given. Returns (y, state_out)."""
    return recur_fwd.__wrapped__(x, decay, rate, gate, scaling, state, None, True, False, out,
                                 state if state_out is None else state_out)


def recur_bwd_workspace_bytes(B: int, T: int, D: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace a recur_bwd of these sizes takes."""
    p = RecurProblem(*_int32("gdn_recur_bwd_workspace_bytes", B, T, D), DTYPES[dtype], *(0,) * 10)
    return _need("gdn_recur_bwd_workspace_bytes", p, _recur_refusal)


def _recur_bwd_plan(dy, x, decay, states, rate, gate, scaling, d_final_state, lengths, dx, d_decay, d_gate,
                    d_rate, d_state):
    _given(dy=dy, states=states)
    p, index = _recur_problem(x, decay, rate, gate, scaling, lengths, dy)
    state, f32 = (x.shape[0], x.shape[2]), torch.float32
    for t, name, form, kind in ((states, "states", _recur_states(x), f32),
                                (d_final_state, "d_final_state", state, f32), (dx, "dx", x.shape, x.dtype),
                                (d_decay, "d_decay", x.shape, x.dtype), (d_gate, "d_gate", x.shape, x.dtype),
                                (d_rate, "d_rate", (x.shape[2],), f32), (d_state, "d_state", state, f32)):
        _dense(t, name, form, kind, index)
    if d_gate is not None and gate is None or d_rate is not None and rate is None:
        raise ValueError("d_gate and d_rate go with a gate and a rate")
    return ctypes.byref(p), state, _need("gdn_recur_bwd_workspace_bytes", p, _recur_refusal), index


def recur_bwd(dy, x, decay, states, rate=None, gate=None, scaling: str = "root", d_final_state=None,
              lengths=None, output_d_state: bool = True, workspace=None, dx=None, d_decay=None, d_gate=None,
              d_rate=None, d_state=None, stream=None):
    """Gradients of recur_fwd (gdn_recur_bwd). Returns (dx, d_decay, d_gate or None, d_rate
    or None, d_state or None), the last for h0.

    dy [B,T,D] in x's dtype, strided, is the gradient of y, ``d_final_state`` [B,D] float32
    that of h_final (None: zeros); ``states`` are those of recur_fwd with
    ``output_states``; the other inputs as given there. ``d_state=d_final_state`` writes in
    place. ``workspace`` (recur_bwd_workspace_bytes) and the gradients may be passed to
    reuse buffers."""
    return _recur_bwd(x, dy, decay, states, rate, gate, scaling, d_final_state, lengths, output_d_state,
                      workspace, dx, d_decay, d_gate, d_rate, d_state, stream=stream)


@_on_stream
def _recur_bwd(x, dy, decay, states, rate, gate, scaling, d_final_state, lengths, output_d_state, workspace, dx,
               d_decay, d_gate, d_rate, d_state):
    key = ("recur_bwd", x.shape, x.stride(), x.dtype, x.get_device(), _form(dy), _form(decay), _form(states),
           _form(rate), _form(gate), scaling, _form(d_final_state), _form(lengths), _form(dx), _form(d_decay),
           _form(d_gate), _form(d_rate), _form(d_state))
    p, state, need, index = _plans.get(key) or _keep(key, _recur_bwd_plan(
        dy, x, decay, states, rate, gate, scaling, d_final_state, lengths, dx, d_decay, d_gate, d_rate, d_state))
    workspace = _workspace(workspace, need, x.device)
    dx = _new(x, lengths) if dx is None else dx
    d_decay = _new(x, lengths) if d_decay is None else d_decay
    if gate is not None and d_gate is None:
        d_gate = _new(x, lengths)
    if rate is not None and d_rate is None:
        d_rate = torch.empty_like(rate)
    if not output_d_state:
        d_state = None
    elif d_state is None:
        d_state = torch.empty(state, dtype=torch.float32, device=x.device)
    _call(lib().gdn_recur_bwd, "gdn_recur_bwd", index, p, dy.data_ptr(), x.data_ptr(), decay.data_ptr(),
          _ptr(gate), _ptr(rate), states.data_ptr(), _ptr(d_final_state), _ptr(lengths), dx.data_ptr(),
          d_decay.data_ptr(), _ptr(d_gate), _ptr(d_rate), _ptr(d_state), workspace.data_ptr(), need)
    return dx, d_decay, d_gate, d_rate, d_state


# -------------------------------------------------------------------- layer norm
def _layer_norm_refusal(p):
    return lib().gdn_layer_norm(ctypes.byref(p), *[None] * 7)


def _layer_norm_problem(x, weight, eps, center, lengths, dy=None):
    """(problem, device index) of the inputs that both passes take."""
    shape, dtype, index = _x(x)
    B, T, C = shape
    p = LayerNormProblem(*_int32("gdn_layer_norm", B, T, C), DTYPES[dtype], 0 if center else GDN_LAYER_NORM_RMS,
                         eps, *_tokens(x, "x", shape, dtype, index), *_optional(dy, "dy", shape, dtype, index))
    _dense(weight, "weight", (C,), torch.float32, index)
    _dense(lengths, "lengths", (B,), torch.int32, index)
    return p, index


def _layer_norm_plan(x, weight, bias, eps, center, lengths, out, stats):
    p, index = _layer_norm_problem(x, weight, eps, center, lengths)
    for t, name, form, kind in ((bias, "bias", (x.shape[2],), torch.float32), (out, "out", x.shape, x.dtype),
                                (stats, "stats", (*x.shape[:2], 2), torch.float32)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), index


@_on_stream
def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, lengths=None,
               output_stats: bool = False, out=None, stats=None):
    """Layer norm of every token's channels (gdn_layer_norm). Returns y, or with
    ``output_stats`` (y, stats):

        y = (x - mean) rstd weight + bias,  rstd = 1 / sqrt(mean((x - mean)^2) + eps)

    with mean = 0 where ``center`` is false (the norm by the root mean square). x [B,T,C]
    float32 or bfloat16, strided; weight, bias [C] float32 or None. ``stats`` [B,T,2]
    float32 (mean, rstd) is what layer_norm_bwd takes. ``out`` may be a contiguous x itself
    (in place)."""
    eps, center = float(eps), bool(center)
    if not output_stats:
        stats = None
    key = ("layer_norm", x.shape, x.stride(), x.dtype, x.get_device(), _form(weight), _form(bias), eps, center,
           _form(lengths), _form(out), _form(stats))
    p, index = _plans.get(key) or _keep(key, _layer_norm_plan(x, weight, bias, eps, center, lengths, out, stats))
    if out is None:
        out = _new(x, lengths)
    if output_stats and stats is None:
        stats = _zeros((*x.shape[:2], 2), torch.float32, x, lengths)
    _call(lib().gdn_layer_norm, "gdn_layer_norm", index, p, x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(lengths),
          out.data_ptr(), _ptr(stats))
    return (out, stats) if output_stats else out


def layer_norm_bwd_workspace_bytes(B: int, T: int, C: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace a layer_norm_bwd of these sizes takes."""
    p = LayerNormProblem(*_int32("gdn_layer_norm_bwd_workspace_bytes", B, T, C), DTYPES[dtype], 0, 0.0, *(0,) * 4)
    return _need("gdn_layer_norm_bwd_workspace_bytes", p, _layer_norm_refusal)


def _layer_norm_bwd_plan(dy, x, stats, weight, center, lengths, dx, d_weight, d_bias):
    _given(dy=dy, stats=stats)
    p, index = _layer_norm_problem(x, weight, 0.0, center, lengths, dy)
    for t, name, form, kind in ((stats, "stats", (*x.shape[:2], 2), torch.float32), (dx, "dx", x.shape, x.dtype),
                                (d_weight, "d_weight", (x.shape[2],), torch.float32),
                                (d_bias, "d_bias", (x.shape[2],), torch.float32)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), _need("gdn_layer_norm_bwd_workspace_bytes", p, _layer_norm_refusal), index


def layer_norm_bwd(dy, x, stats, weight=None, bias: bool = False, center: bool = True, lengths=None,
                   workspace=None, dx=None, d_weight=None, d_bias=None, stream=None):
    """Gradients of layer_norm (gdn_layer_norm_bwd). Returns (dx, d_weight or None, d_bias
    or None): d_weight where a weight is given, d_bias where ``bias`` is true.

    dy [B,T,C] in x's dtype, strided; ``stats`` are those of layer_norm with
    ``output_stats``; x, weight, center and lengths as given there. ``workspace``
    (layer_norm_bwd_workspace_bytes) and the gradients may be passed to reuse buffers."""
    return _layer_norm_bwd(x, dy, stats, weight, bias, center, lengths, workspace, dx, d_weight, d_bias,
                           stream=stream)


@_on_stream
def _layer_norm_bwd(x, dy, stats, weight, bias, center, lengths, workspace, dx, d_weight, d_bias):
    center, C = bool(center), x.shape[-1]
    if d_weight is not None and weight is None or d_bias is not None and not bias:
        raise ValueError("d_weight and d_bias go with a weight and with bias=True")
    key = ("layer_norm_bwd", x.shape, x.stride(), x.dtype, x.get_device(), _form(dy), _form(stats), _form(weight),
           center, _form(lengths), _form(dx), _form(d_weight), _form(d_bias))
    p, need, index = _plans.get(key) or _keep(key, _layer_norm_bwd_plan(
        dy, x, stats, weight, center, lengths, dx, d_weight, d_bias))
    workspace = _workspace(workspace, need, x.device)
    dx = _new(x, lengths) if dx is None else dx
    if weight is not None and d_weight is None:
        d_weight = torch.empty_like(weight)
    if bias and d_bias is None:
        d_bias = torch.empty(C, dtype=torch.float32, device=x.device)
    _call(lib().gdn_layer_norm_bwd, "gdn_layer_norm_bwd", index, p, dy.data_ptr(), x.data_ptr(), stats.data_ptr(),
          _ptr(weight), _ptr(lengths), dx.data_ptr(), _ptr(d_weight), _ptr(d_bias), workspace.data_ptr(), need)
    return dx, d_weight, d_bias


# ------------------------------------------------------------- short convolution
def _conv_bwd_refusal(p):
    return lib().gdn_conv_bwd(ctypes.byref(p), *[None] * 12, 0, None)


def conv_bwd_workspace_bytes(B: int, T: int, C: int, W: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace a conv_bwd of these sizes takes."""
    p = ConvBwdProblem(*_int32("gdn_conv_bwd_workspace_bytes", B, T, C, W), DTYPES[dtype], 0, *(0,) * 4)
    return _need("gdn_conv_bwd_workspace_bytes", p, _conv_bwd_refusal)


def _conv_bwd_plan(dy, x, weight, bias, state, act, d_final_state, lengths, dx, d_weight, d_bias, d_state):
    _given(dy=dy, weight=weight)
    shape, dtype, index = _x(x)
    B, T, C = shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise GdnError(GDN_ERR_UNSUPPORTED, "gdn_conv_bwd")
    window, f32 = (B, W - 1, C), torch.float32
    p = ConvBwdProblem(*_int32("gdn_conv_bwd", B, T, C, W), DTYPES[dtype], _act(act),
                       *_tokens(x, "x", shape, dtype, index), *_tokens(dy, "dy", shape, dtype, index))
    for t, name, form, kind in ((weight, "weight", (C, W), f32), (bias, "bias", (C,), f32),
                                (lengths, "lengths", (B,), torch.int32), (state, "state", window, dtype),
                                (d_final_state, "d_final_state", window, dtype), (dx, "dx", shape, dtype),
                                (d_weight, "d_weight", (C, W), f32), (d_bias, "d_bias", (C,), f32),
                                (d_state, "d_state", window, dtype)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), window, _need("gdn_conv_bwd_workspace_bytes", p, _conv_bwd_refusal), index


def conv_bwd(dy, x, weight, bias=None, state=None, act: str = "silu", d_final_state=None, lengths=None,
             workspace=None, dx=None, d_weight=None, d_bias=None, d_state=None, stream=None):
    """Gradients of conv_fwd (gdn_conv_bwd). Returns (dx, d_weight, d_bias or None, d_state
    or None): d_bias where a bias is given, d_state where a state is.

    dy [B,T,C] in x's dtype, strided, is the gradient of y, ``d_final_state`` [B,W-1,C] in
    x's dtype that of the returned state (None: zeros); the other inputs as given to
    conv_fwd. ``workspace`` (conv_bwd_workspace_bytes) and the gradients may be passed to reuse
    buffers."""
    return _conv_bwd(x, dy, weight, bias, state, act, d_final_state, lengths, workspace, dx, d_weight, d_bias,
                     d_state, stream=stream)


@_on_stream
def _conv_bwd(x, dy, weight, bias, state, act, d_final_state, lengths, workspace, dx, d_weight, d_bias, d_state):
    if d_bias is not None and bias is None or d_state is not None and state is None:
        raise ValueError("d_bias and d_state go with a bias and a state")
    key = ("conv_bwd", x.shape, x.stride(), x.dtype, x.get_device(), _form(dy), _form(weight), _form(bias),
           _form(state), act, _form(d_final_state), _form(lengths), _form(dx), _form(d_weight), _form(d_bias),
           _form(d_state))
    p, window, need, index = _plans.get(key) or _keep(key, _conv_bwd_plan(
        dy, x, weight, bias, state, act, d_final_state, lengths, dx, d_weight, d_bias, d_state))
    workspace = _workspace(workspace, need, x.device)
    dx = _new(x, lengths) if dx is None else dx
    d_weight = torch.empty_like(weight) if d_weight is None else d_weight
    if bias is not None and d_bias is None:
        d_bias = torch.empty_like(bias)
    if state is not None and d_state is None:
        d_state = torch.empty(window, dtype=x.dtype, device=x.device)
    _call(lib().gdn_conv_bwd, "gdn_conv_bwd", index, p, dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
          _ptr(bias), _ptr(state), _ptr(d_final_state), _ptr(lengths), dx.data_ptr(), d_weight.data_ptr(),
          _ptr(d_bias), _ptr(d_state), workspace.data_ptr(), need)
    return dx, d_weight, d_bias, d_state
