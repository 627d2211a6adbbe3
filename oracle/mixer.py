"""fp64 NumPy forms of the operators around the recurrence: the short causal
convolution, the selective state space scan and the group norm (test
infrastructure only; no code shared with the GPU path).

Each function also returns what its error bound needs (see tests/mixer_bounds.py).
Output rows at or past a sequence's length are NaN here.
"""
from __future__ import annotations

import numpy as np


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def act(v, name):
    return {"none": lambda: v, "silu": lambda: v * sigmoid(v), "sigmoid": lambda: sigmoid(v)}[name]()


def clamp_lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def conv(x, weight, bias=None, state=None, lengths=None, act_name="silu"):
    """(y, state, v, S): v the value before the activation, S the sum of its terms' sizes."""
    B, T, C = x.shape
    W = weight.shape[1]
    y, v, S = (np.full((B, T, C), np.nan) for _ in range(3))
    out = np.zeros((B, W - 1, C))
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        seq = np.zeros((W - 1 + n, C))
        if state is not None:
            seq[:W - 1] = state[b]
        seq[W - 1:] = x[b, :n]
        for t in range(n):
            v[b, t] = (0.0 if bias is None else bias) + (seq[t:t + W] * weight.T).sum(0)
            S[b, t] = (0.0 if bias is None else abs(bias)) + abs(seq[t:t + W] * weight.T).sum(0)
        out[b] = seq[n:]
    y = act(v, act_name)
    return y, out, v, S


def softplus(v):
    return np.logaddexp(0.0, v)


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, dt_softplus=False, h0=None, lengths=None,
         unit=2.0 ** -24):
    """(y, h, Ey, Eh): the outputs, and bounds on what fp32 arithmetic of this
    recurrence may be off, carried along it.

    One step's rounding errors, u = 2^-24: v = dt + dt_bias and the softplus of it
    are within (8 + 3|v|) u of Delta (exp's argument |v| log2 e is rounded, its
    result within 2 ulp, the logarithm and sum a few u); the factor exp(Delta A)
    is within 4u + (3u + Delta's) |Delta A|, doubled here for states that cross a
    segment border as exp(A sum Delta); Delta x B takes 3u and Delta's; the sums of
    y take N + 4 roundings of their terms' sizes. Passing one segment's state to
    the next adds the same roundings as a step."""
    B, T, nd = x.shape
    G, N = Bm.shape[2:]
    r = nd // G
    h = np.zeros((B, nd, N)) if h0 is None else h0.astype(np.float64).copy()
    E = np.zeros_like(h)
    y = np.full((B, T, nd), np.nan)
    Ey = np.full((B, T, nd), np.nan)
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        for t in range(n):
            v = dt[b, t] + (0.0 if dt_bias is None else dt_bias)
            step = softplus(v) if dt_softplus else v
            ds = (8 + 3 * abs(v)) * unit if dt_softplus else unit * np.ones_like(v)
            bm, cm = np.repeat(Bm[b, t], r, axis=0), np.repeat(Cm[b, t], r, axis=0)
            sa = step[:, None] * A
            a = np.exp(sa)
            ea = 2 * (4 * unit + (3 * unit + ds[:, None]) * abs(sa))
            term = (step * x[b, t])[:, None] * bm
            E[b] = a * (E[b] + ea * abs(h[b])) + abs(term) * (3 * unit + ds[:, None])
            h[b] = a * h[b] + term
            E[b] += 2 * unit * abs(h[b])
            o = (cm * h[b]).sum(-1)
            skip = 0.0 if D is None else D * x[b, t]
            eo = (abs(cm) * E[b]).sum(-1) + (N + 4) * unit * ((abs(cm * h[b])).sum(-1) + abs(skip))
            o = o + skip
            if z is not None:
                g = act(z[b, t], "silu")
                eo = abs(g) * (eo + abs(o) * (6 + 1.2 * abs(z[b, t])) * 2 * unit) \
                    + abs(o * z[b, t]) * 2.0 ** -126   # a sigmoid below the normal range is 0
                o = o * g
            y[b, t], Ey[b, t] = o, eo
    return y, h, Ey, E


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, act_name="none", gate=None, lengths=None):
    """(y, v, xhat, size): v before the activation, xhat the normalised value, size the
    group's mean of |x| over its deviation (per row, broadcast to x's shape)."""
    B, T, C = x.shape
    v, xhat, size = (np.full((B, T, C), np.nan) for _ in range(3))
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        if n == 0:
            continue
        xb = x[b, :n].reshape(n, groups, C // groups)
        mean = xb.mean((0, 2), keepdims=True)
        sd = np.sqrt(((xb - mean) ** 2).mean((0, 2), keepdims=True) + eps)
        xhat[b, :n] = ((xb - mean) / sd).reshape(n, C)
        size[b, :n] = np.broadcast_to(abs(xb).mean((0, 2), keepdims=True) / sd, xb.shape).reshape(n, C)
    v = xhat * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = v * act(gate, act_name) if gate is not None else act(v, act_name)
    return y, v, xhat, size
