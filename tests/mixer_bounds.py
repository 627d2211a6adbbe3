"""Elementwise error bounds of the mixer operators' tests, from rounding analysis.

u = 2^-24 is fp32's rounding. An output is rounded once to its type, off by at
most eps(type) / 2 of its value. exp(-v) is ex2.approx of -v log2 e: the constant
and the product are rounded, 2u |v| of the result, and PTX states a relative error of
2^-22 = 4u for the instruction; 1 + exp(-v) takes u, rcp.approx 1 ulp, 2u at most,
and the product with v another u. A sigmoid(v) is so off by at most (7 + 2 |v|)u of
itself, v sigmoid(v) by (8 + 2 |v|)u beside the error of v (slope of silu at most 1.1, of
sigmoid 0.25): within the (6 + 1.2 |v|) 2u used here. The quotient 1 / (1 + exp(-v)) is
flushed to 0 below fp32's normal range: what it multiplies is then off by that times
2^-126 at most (TINY)."""
import numpy as np
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126


def act_error(v, ev, y, name):
    """Error of act(v) where v is off by ev."""
    if name == "none":
        return ev
    slope = 1.1 if name == "silu" else 0.25
    return slope * ev + abs(y) * (6 + 1.2 * abs(v)) * 2 * U + np.maximum(1, abs(v)) * TINY


def conv_bound(y, v, S, W, name):
    return act_error(v, (W + 1) * U * S, y, name)


def norm_bound(y, v, xhat, size, weight, name, gate=None, act=None):
    """Sums of a group add at most 256 terms in a row (threads, then trees): the mean
    is off by 256 u mean|x|, the deviation by that relative error of 256 u and a
    root within 2 ulp."""
    w = 1.0 if weight is None else abs(weight)
    ev = w * (256 * U * size + abs(xhat) * (256 * U + 4 * U) + 4 * U * abs(xhat)) + 2 * U * abs(v)
    if gate is None:
        return act_error(v, ev, y, name)
    return abs(act) * ev + abs(y) * (6 + 1.2 * abs(gate)) * 2 * U + abs(v) * np.maximum(1, abs(gate)) * TINY


def check(got, want, bound, dtype, what=""):
    """got (a tensor) within the bound and one rounding of want, where want is a number;
    tiny covers results below the normal range."""
    got = got.detach().cpu().double().numpy()
    at = ~np.isnan(want)
    half = torch.finfo(dtype).eps / 2
    lim = bound + half * (abs(want) + bound) + 1e-35
    assert np.isfinite(got[at]).all(), what
    off = abs(got - want)[at] / lim[at]
    assert off.size == 0 or off.max() <= 1.0, f"{what}: {off.max():.3f} of the bound"


def untouched(got, want, fill):
    """The rows outside the sequences (NaN in want) still hold fill."""
    at = np.isnan(want)
    assert (got.detach().cpu().float().numpy()[at] == fill).all()
