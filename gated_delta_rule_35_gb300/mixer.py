"""The operators around the recurrence in a mixing layer: the short causal
convolution (``conv_fwd``, ``conv_step``), the selective state space scan
(``scan_fwd``, ``scan_step``) and the group norm (``group_norm``).

Like the rest of the binding this file marshals arguments only; the work runs in
the library's kernels on the current stream of the tensors' device, and the
contracts are those of include/gdn.h. Tokens are channels-last; inputs marked
*strided* may be slices of wider tensors (their innermost axes contiguous).
``lengths`` ([B] int32, on the device) holds the valid tokens of each sequence of a
padded batch: rows at or past it are not used, and not written in the outputs (zeros,
then, in an output that the call allocates).
With ``stream`` the call runs, and allocates what it returns, on that stream.
"""
from __future__ import annotations

import ctypes

import torch

from .native import DTYPES, GDN_ERR_UNSUPPORTED, GDN_OK, GdnError, _workspace, lib

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


def _tokens(t, name, shape, dtype, index):
    """Batch and token strides of a strided input [B,T,...]; its innermost axes contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have x's dtype {dtype}")
    if t.shape != shape or t.get_device() != index:
        raise ValueError(f"{name} must be {tuple(shape)} on cuda:{index}")
    st = t.stride()
    if (st[-1] != 1 and shape[-1] > 1) or (len(shape) == 4 and st[2] != shape[3] and shape[2] > 1):
        raise ValueError(f"{name}'s innermost axes must be contiguous")
    return st[:2]


def _dense(t, name, shape, dtype, index):
    """A contiguous tensor, or None."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {tuple(shape)} on cuda:{index}")


def _x(x, axes="[B,T,C]"):
    if not x.is_cuda:
        raise ValueError("inputs must be CUDA tensors")
    if x.dtype not in DTYPES:
        raise TypeError("x must be float32 or bfloat16")
    if x.dim() != 3:
        raise ValueError(f"x must be {axes}")
    return x.shape, x.dtype, x.get_device()


def _int32(what, *sizes):
    """The sizes, refused where a problem's 32-bit field would wrap one."""
    if any(not -2 ** 31 <= n < 2 ** 31 for n in sizes):
        raise GdnError(GDN_ERR_UNSUPPORTED, what)
    return sizes


def _act(act):
    a = ACTS.get(act)
    if a is None:
        raise ValueError(f"act must be one of {', '.join(ACTS)}")
    return a


def _new(x, lengths):
    """An output of x's form; of a padded batch zeros, since some rows stay unwritten."""
    return (torch.empty if lengths is None else torch.zeros)(x.shape, dtype=x.dtype, device=x.device)


def _call(f, what, index, *args):
    """f(*args, stream) on device ``index`` and its current stream."""
    s = torch._C._cuda_getCurrentRawStream(index)    # current_stream(index).cuda_stream, 1.9 us sooner
    if index == torch.cuda.current_device():
        st = f(*args, s)
    else:
        with torch.cuda.device(index):
            st = f(*args, s)
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


def _form(t):
    """What a call checks of a tensor: two tensors of one form pass or fail alike."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


# The checked problem of each form of call (as the host entry keeps its plans): checking a
# scan's eleven tensors again would cost a single token 5 us.
_plans: dict = {}


def _keep(key, plan):
    if len(_plans) >= 512:
        _plans.clear()
    _plans[key] = plan
    return plan


def _conv_plan(x, weight, bias, state, lengths, act, out, final_state):
    """(problem, shape of the window state, device index), or the refusal."""
    shape, dtype, index = _x(x)
    B, T, C = shape
    if weight.dim() != 2:
        raise ValueError("weight must be [C,W]")
    W = weight.shape[1]
    if not 2 <= W <= 4:
        raise GdnError(GDN_ERR_UNSUPPORTED, "gdn_conv_fwd")
    window = (B, W - 1, C)
    p = ConvProblem(*_int32("gdn_conv_fwd", B, T, C, W), DTYPES[dtype], _act(act),
                    *_tokens(x, "x", shape, dtype, index))
    for t, name, form, kind in ((weight, "weight", (C, W), torch.float32), (bias, "bias", (C,), torch.float32),
                                (lengths, "lengths", (B,), torch.int32), (state, "state", window, dtype),
                                (out, "out", shape, dtype), (final_state, "final_state", window, dtype)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), window, index


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
    key = (x.shape, x.stride(), x.dtype, x.get_device(), weight.shape, weight.stride(), weight.dtype,
           weight.get_device(), _form(bias), _form(state), _form(lengths), _form(out), _form(final_state),
           act)
    p, window, index = _plans.get(key) or _keep(key, _conv_plan(
        x, weight, bias, state, lengths, act, out, final_state))
    if out is None:
        out = _new(x, lengths)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty(window, dtype=x.dtype, device=x.device)
    _call(lib().gdn_conv_fwd, "gdn_conv_fwd", index, p, x.data_ptr(), weight.data_ptr(), _ptr(bias),
          _ptr(state), _ptr(lengths), out.data_ptr(), _ptr(final_state))
    return out, final_state


@_on_stream
def conv_step(x, weight, state, bias=None, act: str = "silu", state_out=None, out=None):
    """conv_fwd for the next token(s) of every sequence: advances ``state``
    [B,W-1,C] by x's T tokens, in place unless ``state_out`` is given. Returns (y,
    state_out)."""
    return conv_fwd.__wrapped__(x, weight, bias, state, None, act, True, out,
                                state if state_out is None else state_out)


_INVALID = ctypes.c_size_t(-1).value


def scan_workspace_bytes(B: int, T: int, D: int, N: int, G: int = 1, dtype=torch.bfloat16) -> int:
    """Bytes of workspace a scan_fwd of these sizes takes (0: none)."""
    sizes = _int32("gdn_scan_workspace_bytes", B, T, D, N, G)
    p = ScanProblem(*sizes, DTYPES[dtype], 0, 0, *(0,) * 10)
    need = lib().gdn_scan_workspace_bytes(ctypes.byref(p))
    if need == _INVALID:
        raise GdnError(_refusal(p), "gdn_scan_workspace_bytes")
    return need


def _refusal(p) -> int:
    """The status of a problem that the library refuses before any pointer."""
    return lib().gdn_scan_fwd(ctypes.byref(p), *[None] * 13, 0, None)


def _scan_plan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, lengths, out, final_state):
    """(problem, workspace bytes, shape of the state, device index), or the refusal."""
    shape, dtype, index = _x(x, "[B,T,D]")
    nb, T, nd = shape
    if B.dim() != 4:
        raise ValueError("B and C must be [B,T,G,N]")
    G, N = B.shape[2:]
    rows, state, f32 = (nb, T, G, N), (nb, nd, N), torch.float32
    p = ScanProblem(*_int32("gdn_scan_fwd", nb, T, nd, N, G), DTYPES[dtype],
                    GDN_SCAN_SOFTPLUS if dt_softplus else 0, 0,
                    *_tokens(x, "x", shape, dtype, index), *_tokens(dt, "dt", shape, dtype, index),
                    *((0, 0) if z is None else _tokens(z, "z", shape, dtype, index)),
                    *_tokens(B, "B", rows, dtype, index), *_tokens(C, "C", rows, dtype, index))
    for t, name, form, kind in ((A, "A", (nd, N), f32), (D, "D", (nd,), f32), (dt_bias, "dt_bias", (nd,), f32),
                                (h0, "h0", state, f32), (lengths, "lengths", (nb,), torch.int32),
                                (out, "out", shape, dtype), (final_state, "final_state", state, f32)):
        _dense(t, name, form, kind, index)
    need = lib().gdn_scan_workspace_bytes(ctypes.byref(p))
    if need == _INVALID:
        raise GdnError(_refusal(p), "gdn_scan_fwd")
    return ctypes.byref(p), need, state, index


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
    key = (x.shape, x.stride(), x.dtype, x.get_device(), dt.shape, dt.stride(), dt.dtype, dt.get_device(),
           A.shape, A.stride(), A.dtype, A.get_device(), B.shape, B.stride(), B.dtype, B.get_device(),
           C.shape, C.stride(), C.dtype, C.get_device(), _form(D), _form(z), _form(dt_bias), _form(h0),
           _form(lengths), _form(out), _form(final_state), bool(dt_softplus))
    p, need, state, index = _plans.get(key) or _keep(key, _scan_plan(
        x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, lengths, out, final_state))
    if need:    # held until the call: freed before, out could be allocated in its place
        workspace = _workspace(workspace, need, x.device)
    if out is None:
        out = _new(x, lengths)
    if not output_final_state:
        final_state = None
    elif final_state is None:
        final_state = torch.empty(state, dtype=torch.float32, device=x.device)
    _call(lib().gdn_scan_fwd, "gdn_scan_fwd", index, p, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
          B.data_ptr(), C.data_ptr(), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), _ptr(lengths),
          out.data_ptr(), _ptr(final_state), _ptr(workspace) if need else None, need)
    return out, final_state


@_on_stream
def scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus: bool = False,
              state_out=None, out=None):
    """scan_fwd for the next token(s) of every sequence: advances ``state`` [B,D,N]
    float32 by x's T tokens, in place unless ``state_out`` is given. Returns (y,
    state_out)."""
    return scan_fwd.__wrapped__(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, None, True, None,
                                out, state if state_out is None else state_out)


def _norm_plan(x, groups, weight, bias, eps, act, gate, lengths, out):
    """(problem, device index), or the refusal."""
    shape, dtype, index = _x(x)
    B, T, C = shape
    p = GroupNormProblem(*_int32("gdn_group_norm", B, T, C, groups), DTYPES[dtype], _act(act), eps, 0,
                         *_tokens(x, "x", shape, dtype, index),
                         *((0, 0) if gate is None else _tokens(gate, "gate", shape, dtype, index)))
    for t, name, form, kind in ((weight, "weight", (C,), torch.float32), (bias, "bias", (C,), torch.float32),
                                (lengths, "lengths", (B,), torch.int32), (out, "out", shape, dtype)):
        _dense(t, name, form, kind, index)
    return ctypes.byref(p), index


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
    groups, eps = int(groups), float(eps)
    key = (x.shape, x.stride(), x.dtype, x.get_device(), groups, _form(weight), _form(bias), eps, act,
           _form(gate), _form(lengths), _form(out))
    p, index = _plans.get(key) or _keep(key, _norm_plan(x, groups, weight, bias, eps, act, gate, lengths, out))
    if out is None:
        out = _new(x, lengths)
    _call(lib().gdn_group_norm, "gdn_group_norm", index, p, x.data_ptr(), _ptr(weight), _ptr(bias),
          _ptr(gate), _ptr(lengths), out.data_ptr())
    return out
