"""The operators around the recurrence in a mixing layer: the short causal
convolution (``conv_fwd``, ``conv_step``), the selective state space scan
(``scan_fwd``, ``scan_step``) and the group norm (``group_norm``).

Like the rest of the binding this file marshals arguments only; the work runs in
the library's kernels on the current stream of the tensors' device, and the
contracts are those of include/gdn.h. Tokens are channels-last; inputs marked
*strided* may be slices of wider tensors (their innermost axes contiguous).
``lengths`` ([B] int32, on the device) holds the valid tokens of each sequence of a
padded batch: rows at or past it are not used, and not written in the outputs.
With ``stream`` the call runs, and allocates what it returns, on that stream.
"""
from __future__ import annotations

import ctypes

import torch

from .native import DTYPES, GDN_ERR_UNSUPPORTED, GDN_OK, GdnError, _given, _workspace, lib

ACTS = {"none": 0, "silu": 1, "sigmoid": 2}
GDN_SCAN_SOFTPLUS = 1


class ConvProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "W", "dtype", "act")] + \
               [(n, ctypes.c_int64) for n in ("x_stride_b", "x_stride_t")]


class ScanProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "N", "G", "dtype", "flags", "reserved")] + \
               [(f"{n}_stride_{a}", ctypes.c_int64) for n in ("x", "dt", "z", "b", "c") for a in "bt"]


class GroupNormProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "C", "G", "dtype", "act")] + \
               [("eps", ctypes.c_float), ("reserved", ctypes.c_int32)] + \
               [(f"{n}_stride_{a}", ctypes.c_int64) for n in ("x", "gate") for a in "bt"]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _tokens(t, name, shape, like):
    """A strided input: the innermost axes (all but batch and tokens) contiguous."""
    if t.dtype != like.dtype:
        raise TypeError(f"{name} must have x's dtype {like.dtype}")
    if t.shape != shape or t.device != like.device:
        raise ValueError(f"{name} must be {tuple(shape)} on {like.device}")
    inner = 1
    for n, s in zip(reversed(shape[2:]), reversed(t.stride()[2:])):
        if n > 1 and s != inner:
            raise ValueError(f"{name}'s innermost axes must be contiguous")
        inner *= n
    return t.stride()[:2]


def _weights(t, name, shape, dev):
    if t is None:
        return None
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32")
    if t.shape != shape or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)} on {dev}")
    return t.data_ptr()


def _lengths(t, B, dev):
    if t is None:
        return None
    if t.dtype != torch.int32:
        raise TypeError("lengths must be int32")
    if t.shape != (B,) or t.device != dev or not t.is_contiguous():
        raise ValueError(f"lengths must be contiguous ({B},) on {dev}")
    return t.data_ptr()


def _x(x, axes="[B,T,C]"):
    if x.device.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    if x.dtype not in DTYPES:
        raise TypeError("x must be float32 or bfloat16")
    if x.dim() != 3:
        raise ValueError(f"x must be {axes}")
    return x.shape


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return ACTS[act]


def _call(f, what, dev, *args):
    """f(*args, stream) on the tensors' device and its current stream."""
    s = torch.cuda.current_stream(dev)
    if dev.index == torch.cuda.current_device():
        st = f(*args, s.cuda_stream)
    else:
        with torch.cuda.device(dev):
            st = f(*args, s.cuda_stream)
    if st != GDN_OK:
        raise GdnError(st, what)


def _on_stream(f):
    """Runs f with ``stream`` current, so that what it allocates belongs to it."""
    def call(x, *args, stream=None, **kw):
        if stream is None:
            return f(x, *args, **kw)
        if stream.device != x.device:
            raise ValueError("stream must belong to the tensors' device")
        with torch.cuda.stream(stream):
            return f(x, *args, **kw)
    call.__name__, call.__doc__, call.__wrapped__ = f.__name__, f.__doc__, f
    return call


@_on_stream
def conv_fwd(x, weight, bias=None, state=None, lengths=None, act: str = "silu",
             output_final_state: bool = True, out=None, final_state=None):
    """Causal depthwise convolution over tokens (gdn_conv_fwd). Returns (y, state
    or None):

        y[b,t,c] = act(bias[c] + sum_k weight[c,k] x[b, t - W + 1 + k, c])

    x [B,T,C] float32 or bfloat16, strided; weight [C,W], W in 2..4, and bias [C]
    float32; ``state`` [B,W-1,C] in x's dtype: the last inputs before the first
    token (None: zeros). The returned state holds the last W-1 inputs up to the
    last valid token; ``final_state=state`` updates it in place. ``act``: "silu",
    "none" or "sigmoid". ``out`` [B,T,C] may be passed to reuse a buffer."""
    B, T, C = _x(x)
    dev = x.device
    sb, st = _tokens(x, "x", x.shape, x)
    if weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise GdnError(GDN_ERR_UNSUPPORTED, "gdn_conv_fwd")
    shape = (B, W - 1, C)
    p = ConvProblem(B, T, C, W, DTYPES[x.dtype], _act(act), sb, st)
    w = _weights(weight, "weight", (C, W), dev)
    bi = _weights(bias, "bias", (C,), dev)
    n = _lengths(lengths, B, dev)
    if state is not None:
        _given(state, shape, x.dtype, dev, "state")
    y = torch.empty((B, T, C), dtype=x.dtype, device=dev) if out is None else \
        _given(out, (B, T, C), x.dtype, dev, "out")
    so = None
    if output_final_state:
        so = torch.empty(shape, dtype=x.dtype, device=dev) if final_state is None else \
            _given(final_state, shape, x.dtype, dev, "final_state")
    _call(lib().gdn_conv_fwd, "gdn_conv_fwd", dev, ctypes.byref(p), x.data_ptr(), w, bi,
          _ptr(state), n, y.data_ptr(), _ptr(so))
    return y, so


def conv_step(x, weight, state, bias=None, act: str = "silu", state_out=None, out=None, stream=None):
    """conv_fwd for the next token(s) of every sequence: advances ``state``
    [B,W-1,C] by x's T tokens, in place unless ``state_out`` is given. Returns (y,
    state_out)."""
    return conv_fwd(x, weight, bias, state, act=act, out=out,
                    final_state=state if state_out is None else state_out, stream=stream)


def _scan_problem(B, T, D, N, G, dtype, flags=0, strides=(0,) * 10):
    return ScanProblem(B, T, D, N, G, DTYPES[dtype], flags, 0, *strides)


def scan_workspace_bytes(B: int, T: int, D: int, N: int, G: int = 1, dtype=torch.bfloat16) -> int:
    """Bytes of workspace a scan_fwd of these sizes takes (0: none)."""
    p = _scan_problem(B, T, D, N, G, dtype)
    need = int(lib().gdn_scan_workspace_bytes(ctypes.byref(p)))
    if need == ctypes.c_size_t(-1).value:
        raise GdnError(_refusal(p), "gdn_scan_workspace_bytes")
    return need


def _refusal(p) -> int:
    """The status of a problem that the library refuses before any pointer."""
    return lib().gdn_scan_fwd(ctypes.byref(p), *[None] * 13, 0, None)


@_on_stream
def scan_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False, h0=None,
             lengths=None, output_final_state: bool = True, workspace=None, out=None,
             final_state=None):
    """Selective state space scan (gdn_scan_fwd). Returns (y, h_final or None):

        Delta = softplus(dt + dt_bias)          (dt + dt_bias without dt_softplus)
        h[d,n] <- exp(Delta[d] A[d,n]) h[d,n] + Delta[d] x[d] B[g,n]
        y[d] = (sum_n C[g,n] h[d,n] + D[d] x[d]) * silu(z[d])

    per token, g = d // (D/G). x, dt, z [B,T,D] and B, C [B,T,G,N] float32 or
    bfloat16 (one dtype), strided; A [D,N], D and dt_bias [D], h0 and h_final
    [B,D,N] float32; N in 1..128. ``final_state=h0`` updates the state in place.
    ``workspace`` (scan_workspace_bytes) and ``out`` may be passed to reuse
    buffers."""
    nb, T, nd = _x(x, "[B,T,D]")
    dev = x.device
    if B.dim() != 4:
        raise ValueError("B and C must be [B,T,G,N]")
    G, N = B.shape[2:]
    strides = _tokens(x, "x", x.shape, x) + _tokens(dt, "dt", x.shape, x)
    strides += (0, 0) if z is None else _tokens(z, "z", x.shape, x)
    strides += _tokens(B, "B", (nb, T, G, N), x) + _tokens(C, "C", (nb, T, G, N), x)
    p = _scan_problem(nb, T, nd, N, G, x.dtype, GDN_SCAN_SOFTPLUS if dt_softplus else 0, strides)
    a = _weights(A, "A", (nd, N), dev)
    skip, bias = _weights(D, "D", (nd,), dev), _weights(dt_bias, "dt_bias", (nd,), dev)
    hi = _weights(h0, "h0", (nb, nd, N), dev)
    n = _lengths(lengths, nb, dev)
    need = int(lib().gdn_scan_workspace_bytes(ctypes.byref(p)))
    if need == ctypes.c_size_t(-1).value:
        raise GdnError(_refusal(p), "gdn_scan_fwd")
    if need:
        workspace = _workspace(workspace, need, dev)
    y = torch.empty((nb, T, nd), dtype=x.dtype, device=dev) if out is None else \
        _given(out, (nb, T, nd), x.dtype, dev, "out")
    hf = None
    if output_final_state:
        hf = torch.empty((nb, nd, N), dtype=torch.float32, device=dev) if final_state is None else \
            _given(final_state, (nb, nd, N), torch.float32, dev, "final_state")
    _call(lib().gdn_scan_fwd, "gdn_scan_fwd", dev, ctypes.byref(p), x.data_ptr(),
          dt.data_ptr(), a, B.data_ptr(), C.data_ptr(), skip, _ptr(z), bias, hi, n, y.data_ptr(),
          _ptr(hf), _ptr(workspace) if need else None, need)
    return y, hf


def scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
              state_out=None, out=None, stream=None):
    """scan_fwd for the next token(s) of every sequence: advances ``state`` [B,D,N]
    float32 by x's T tokens, in place unless ``state_out`` is given. Returns (y,
    state_out)."""
    return scan_fwd(x, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus, h0=state,
                    out=out, final_state=state if state_out is None else state_out, stream=stream)


@_on_stream
def group_norm(x, groups: int, weight=None, bias=None, eps: float = 1e-5, act: str = "none",
               gate=None, lengths=None, out=None):
    """Group norm of channels-last rows with an activation (gdn_group_norm): mean and
    variance over a sequence's valid tokens and the C / groups channels of a group,

        v = (x - mean) / sqrt(var + eps) * weight + bias
        y = act(v), or v * act(gate) with a gate

    x and gate [B,T,C] float32 or bfloat16, strided; weight, bias [C] float32 or
    None. For the norm of every token on its own pass x as [tokens,1,C]. ``out``
    may be a contiguous x itself (in place)."""
    B, T, C = _x(x)
    dev = x.device
    strides = _tokens(x, "x", x.shape, x)
    strides += (0, 0) if gate is None else _tokens(gate, "gate", x.shape, x)
    p = GroupNormProblem(B, T, C, int(groups), DTYPES[x.dtype], _act(act), float(eps), 0, *strides)
    w, bi = _weights(weight, "weight", (C,), dev), _weights(bias, "bias", (C,), dev)
    n = _lengths(lengths, B, dev)
    y = torch.empty((B, T, C), dtype=x.dtype, device=dev) if out is None else \
        _given(out, (B, T, C), x.dtype, dev, "out")
    _call(lib().gdn_group_norm, "gdn_group_norm", dev, ctypes.byref(p), x.data_ptr(), w, bi,
          _ptr(gate), n, y.data_ptr())
    return y
