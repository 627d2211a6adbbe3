"""fp64 NumPy forms of the gated linear recurrence, layer norm and the short convolution
with their gradients (test infrastructure only; no code shared with the GPU path).

Each function returns a dict of values and a dict, with the same names, of bounds on what
fp32 arithmetic of these formulas may be off before an output's own rounding. Rows at or
past a sequence's length are NaN in the values.

The bounds, u = 2^-24 fp32's rounding and tiny = 2^-126 the end of its normal range:

* exp(-v) by the exp2 instruction is off by (4 + 2 |v|) u of itself (its argument's constant
  and product are rounded, the instruction is within 4u), a reciprocal by 2u: sigmoid(v) is
  so off by (7 + 2 |v|) u of itself, 1 - sigmoid(v) as exp(-v) sigmoid(v) by (12 + 4 |v|) u;
  either by tiny where it is below the normal range. |v| counts up to FAR: from there on both
  are 0 or 1 but for tiny.
* a = exp(g) with g off by eg of itself: a is off by a (eg |g| + 2u |g| + 4u), and by tiny where
  it is below the normal range; 1 - a, with a |g| <= 1 - a, by (eg + 6u) of itself.
* Sums along the tokens are bounded with the sum of their terms' sizes, M <- a M + |u|, in
  place of the state, so that the bound holds for any order in which the terms are
  added up: a token adds the error of its factor twice (in the state and in a product of
  factors) and 4u M.
* A sum over tokens or channels takes at most SUMS additions in a row. `additions` counts those of a sum
  over tokens; the forms are compared at sizes where it gives no more, and a larger one is
  bounded with its own count."""
from __future__ import annotations

import math

import numpy as np

from .mixer import clamp_lengths, sigmoid

U = 2.0 ** -24
TINY = 2.0 ** -126
SUMS = 600
FAR = 150.0
# What a sigmoid off by tiny makes of sqrt(1 - a^2) <= sqrt(2 rate s), of rate s / sqrt(2 rate s) and of
# s / sqrt(2 rate s), for rates of 0.002 to 300.
SMALL = 2.0 ** -58


def additions(terms, parts):
    """Additions in a row of a sum over tokens of which a thread adds `terms` in turn, and which leaves
    `parts` partial results: these go eight and more to a thread, 32 threads at most to a sum, and on in a
    tree. `terms` is, for the rate's gradient, a lane's share of a sequence (its tokens over the warps of its
    cluster, up to a tile, and the warps); for the norm's, a block's share of the rows (of 304 blocks, of 152
    where one fills an SM, of 64 where a row is more than a block holds) and the rows it holds at once; for the
    convolution's, a run of 256 tokens at most and the runs of a block."""
    return math.ceil(terms) + max(8, math.ceil(parts / 32)) + 5


def sigmoids(v):
    """sigmoid(v), 1 - it and the relative errors of both."""
    size = np.minimum(abs(v), FAR)
    return sigmoid(v), sigmoid(-v), (7 + 2 * size) * U, (12 + 4 * size) * U


def factors(decay, gate, rate, scaling):
    """Of all tokens, as a dict; names that begin with e are relative errors."""
    s, sn, es, esn = sigmoids(decay)
    if rate is None:
        a, an, ea, ean = s, sn, es, esn
    else:
        g = rate * s
        eg = es + U
        a, an = np.exp(-g), -np.expm1(-g)
        ea, ean = (eg + 2 * U) * g + 4 * U, eg + 6 * U
    if scaling == "root":
        v = an * (1 + a)
        m = np.sqrt(v)
        em = (ean + ea) / 2 + 8 * U
        with np.errstate(divide="ignore", invalid="ignore"):
            ml = np.where(v > 0, -a * a / m, 0.0)
        eml = 2 * ea + em + 2 * U
    elif scaling == "complement":
        m, em, ml, eml = an, ean, -a, ea
    else:
        m, em, ml, eml = np.ones_like(a), 0.0, np.zeros_like(a), 0.0
    q, qn, eq, eqn = (np.ones_like(a), np.zeros_like(a), 0.0, 0.0) if gate is None else sigmoids(gate)
    return dict(s=s, sn=sn, es=es, esn=esn, a=a, an=an, ea=ea, ean=ean, m=m, em=em, ml=ml, eml=eml, q=q, qn=qn,
                eq=eq, eqn=eqn)


def recur(x, decay, rate=None, gate=None, scaling="root", h0=None, lengths=None, every=16):
    """({y, h, states}, bounds, {before, M, E}): the state before each token, the size and the
    error that it carries."""
    B, T, D = x.shape
    K = (T + every - 1) // every
    y, before, M, E, Ey = (np.full((B, T, D), np.nan) for _ in range(5))
    states, Es = np.full((B, K, D), np.nan), np.full((B, K, D), np.nan)
    h = np.zeros((B, D)) if h0 is None else h0.copy()
    eh = np.zeros((B, D))
    f = factors(decay, gate, rate, scaling)
    with np.errstate(invalid="ignore"):
        u = f["m"] * f["q"] * x
        eu = abs(u) * (f["em"] + f["eq"] + 3 * U) + abs(x) * (
            SMALL if scaling == "root" else TINY * (1.0 if rate is None else np.maximum(rate, 1)))
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        size, err = abs(h[b]), eh[b]
        for t in range(n):
            if t % every == 0:
                states[b, t // every], Es[b, t // every] = h[b], err
            before[b, t], M[b, t], E[b, t] = h[b], size, err
            a, ea = f["a"][b, t], f["ea"][b, t] * np.ones(D)
            err = a * (err + 2 * ea * size) + eu[b, t] + TINY * size
            size = a * size + abs(u[b, t])
            err = err + 4 * U * size
            h[b] = a * h[b] + u[b, t]
            y[b, t], Ey[b, t] = h[b], err
        eh[b] = err
    return dict(y=y, h=h, states=states), dict(y=Ey, h=eh, states=Es), dict(before=before, M=M, E=E)


def recur_bwd(dy, x, decay, rate=None, gate=None, scaling="root", h0=None, d_final=None, lengths=None, every=16):
    """({dx, d_decay, d_gate, d_rate, d_state}, bounds), the states being those of recur."""
    B, T, D = x.shape
    f = factors(decay, gate, rate, scaling)
    kept = recur(x, decay, rate, gate, scaling, h0, lengths, every)[2]
    lam, el = np.full((B, T, D), np.nan), np.full((B, T, D), np.nan)
    first, ef = np.zeros((B, D)), np.zeros((B, D))
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        carry = np.zeros(D) if d_final is None else d_final[b].copy()
        size, err = abs(carry), np.zeros(D)
        for t in range(n - 1, -1, -1):
            a, ea = f["a"][b, t], f["ea"][b, t] * np.ones(D)
            size = size + abs(dy[b, t])
            err = err + 4 * U * size
            lam[b, t], el[b, t] = dy[b, t] + carry, err
            carry = a * lam[b, t]
            err = a * (err + 2 * ea * size) + TINY * size
            size = a * size
        first[b], ef[b] = carry, err + 2 * U * size
    m, q, s, sn, a = (f[k] for k in ("m", "q", "s", "sn", "a"))
    times = 1.0 if rate is None else np.maximum(rate, 1)       # rate s is off by rate tiny
    small = SMALL if scaling == "root" else TINY * times       # of a factor m below the normal range
    dx = lam * m * q
    out = dict(dx=dx, d_gate=None, d_rate=None, d_state=first)
    bound = dict(dx=m * q * el + abs(dx) * (f["em"] + f["eq"] + 3 * U) + abs(lam) * small, d_state=ef)
    if gate is not None:
        out["d_gate"] = dg = dx * x * f["qn"]
        bound["d_gate"] = m * q * f["qn"] * abs(x) * el + abs(dg) * (f["em"] + f["eq"] + f["eqn"] + 5 * U) \
            + abs(lam * x) * (small + TINY)
    first_part, second = a * kept["before"], q * x * f["ml"]
    inner = first_part + second
    ei = a * kept["E"] + abs(first_part) * f["ea"] + abs(second) * (f["eq"] + f["eml"] + 3 * U) \
        + 2 * U * (abs(first_part) + abs(second)) + TINY * kept["M"]
    dlog = lam * inner
    edl = abs(lam) * ei + el * (abs(inner) + ei) + abs(dlog) * U
    root = abs(lam * q * x) * SMALL * (scaling == "root")
    if rate is None:
        slope, esl = f["an"], f["ean"]
    else:
        slope, esl = -rate * s * sn, f["es"] + f["esn"] + 3 * U
        terms = -dlog * s
        live = ~np.isnan(terms)
        total = np.where(live, abs(terms), 0).sum((0, 1))
        out["d_rate"] = np.where(live, terms, 0).sum((0, 1))
        bound["d_rate"] = np.where(live, edl * s + abs(terms) * (f["es"] + U) + root, 0).sum((0, 1)) + SUMS * U * total
    out["d_decay"] = dlog * slope
    bound["d_decay"] = edl * abs(slope) + abs(out["d_decay"]) * (esl + U) \
        + abs(lam) * (abs(first_part) + abs(second) * (scaling != "root")) * TINY * times + root
    return out, bound


def norm_parts(x, eps, center):
    """(xhat, its error, mean, its error, rstd, its relative error) of every token."""
    mean = x.mean(-1, keepdims=True) if center else np.zeros_like(x[..., :1])
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    emean = 256 * U * abs(x).mean(-1, keepdims=True) if center else 0 * mean
    # the deviations' errors are the mean's; SUMS / 2 additions, the root and its argument
    with np.errstate(invalid="ignore"):
        er = (SUMS / 2 + 8) * U + emean ** 2 * rstd ** 2
    xhat = (x - mean) * rstd
    return xhat, rstd * (emean + U * abs(x - mean)) + abs(xhat) * (er + U), mean, emean, rstd, er


def layer_norm(x, weight=None, bias=None, eps=1e-5, center=True, lengths=None):
    """({y, stats}, bounds)."""
    B, T, C = x.shape
    xhat, ex, mean, em, rstd, er = norm_parts(x, eps, center)
    w = 1.0 if weight is None else weight
    y = xhat * w + (0.0 if bias is None else bias)
    stats, es = np.concatenate([mean, rstd], -1), np.concatenate([em, rstd * er], -1)
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        y[b, n:] = stats[b, n:] = np.nan
    return dict(y=y, stats=stats), dict(y=abs(w) * ex + U * abs(xhat * w) + U * abs(y), stats=es)


def layer_norm_bwd(dy, x, weight=None, eps=1e-5, center=True, lengths=None):
    """({dx, d_weight, d_bias}, bounds)."""
    B, T, C = x.shape
    xhat, ex, _, _, rstd, er = norm_parts(x, eps, center)
    v = dy * (1.0 if weight is None else weight)
    c1 = v.mean(-1, keepdims=True) if center else 0.0
    c2 = (v * xhat).mean(-1, keepdims=True)
    e1 = (SUMS / 2) * U * abs(v).mean(-1, keepdims=True) if center else 0.0
    e2 = (SUMS / 2 + 2) * U * abs(v * xhat).mean(-1, keepdims=True) + (abs(v) * ex).mean(-1, keepdims=True)
    dx = rstd * (v - c1 - xhat * c2)
    edx = rstd * (U * abs(v) + e1 + abs(xhat) * e2 + ex * (abs(c2) + e2)
                  + 4 * U * (abs(v) + abs(c1) + abs(xhat * c2))) + abs(dx) * (er + U)
    dw, db, edw, edb = (np.zeros(C) for _ in range(4))
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        dx[b, n:] = np.nan
        dw += (dy * xhat)[b, :n].sum(0)
        db += dy[b, :n].sum(0)
        edw += (abs(dy) * ex + SUMS * U * abs(dy * xhat))[b, :n].sum(0)
        edb += SUMS * U * abs(dy[b, :n]).sum(0)
    return dict(dx=dx, d_weight=dw, d_bias=db), dict(dx=edx, d_weight=edw, d_bias=edb)


def conv_bwd(dy, x, weight, bias=None, state=None, act_name="silu", d_final=None, lengths=None):
    """({dx, d_weight, d_bias, d_state}, bounds)."""
    B, T, C = x.shape
    W = weight.shape[1]
    dx, edx = np.full((B, T, C), np.nan), np.full((B, T, C), np.nan)
    ds, eds = np.zeros((B, W - 1, C)), np.zeros((B, W - 1, C))
    dw, edw, db, edb = np.zeros((C, W)), np.zeros((C, W)), np.zeros(C), np.zeros(C)
    for b, n in enumerate(clamp_lengths(lengths, B, T)):
        seq = np.zeros((W - 1 + n, C))
        if state is not None:
            seq[:W - 1] = state[b]
        seq[W - 1:] = x[b, :n]
        taps = np.stack([seq[k:k + n] for k in range(W)], -1)              # [n, C, W]
        v = (taps * weight).sum(-1) + (0.0 if bias is None else bias)
        ev = (W + 1) * U * (abs(taps * weight).sum(-1) + (0.0 if bias is None else abs(bias)))
        s, sn, es, esn = sigmoids(v)
        if act_name == "none":
            slope, esl = np.ones_like(v), np.zeros_like(v)
        elif act_name == "silu":        # |silu''| <= 1/2
            slope = s * (1 + v * sn)
            esl = 0.5 * ev + s * (1 + abs(v) * sn) * (es + esn + 3 * U) + np.maximum(1, abs(v)) * TINY
        else:                           # |sigmoid''| <= 0.1
            slope, esl = s * sn, 0.1 * ev + s * sn * (es + esn + U) + TINY
        p = dy[b, :n] * slope
        ep = abs(dy[b, :n]) * esl + U * abs(p)
        g, eg = np.zeros_like(seq), np.zeros_like(seq)
        for k in range(W):
            g[k:k + n] += p * weight[:, k]
            eg[k:k + n] += abs(weight[:, k]) * (ep + (W + 2) * U * abs(p))
            dw[:, k] += (p * taps[..., k]).sum(0)
            edw[:, k] += (ep * abs(taps[..., k]) + SUMS * U * abs(p * taps[..., k])).sum(0)
        if d_final is not None:
            g[n:] += d_final[b]
            eg[n:] += 2 * U * abs(d_final[b])
        db += p.sum(0)
        edb += (ep + SUMS * U * abs(p)).sum(0)
        ds[b], eds[b] = g[:W - 1], eg[:W - 1]
        dx[b, :n], edx[b, :n] = g[W - 1:], eg[W - 1:]
    return dict(dx=dx, d_weight=dw, d_bias=db, d_state=ds), dict(dx=edx, d_weight=edw, d_bias=edb, d_state=eds)
