"""The convolution's, scan's and group norm's C entries and wrappers refuse bad calls
before touching CUDA."""
import ctypes

import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import mixer, native

INVALID, UNSUPPORTED = native.GDN_ERR_INVALID_ARG, native.GDN_ERR_UNSUPPORTED
ALIGNMENT, WORKSPACE = native.GDN_ERR_ALIGNMENT, native.GDN_ERR_WORKSPACE


def fake(i):
    """Aligned non-NULL addresses 16 GiB apart; never dereferenced by validation."""
    return (i + 1) << 34


CONV_ARGS = ("x", "weight", "bias", "state_in", "lengths", "y", "state_out")
SCAN_ARGS = ("x", "dt", "A", "Bm", "Cm", "skip", "z", "dt_bias", "h0", "lengths", "y", "h_final",
             "workspace")
NORM_ARGS = ("x", "weight", "bias", "gate", "lengths", "y")


def pointers(names, over):
    ptr = {n: fake(i) for i, n in enumerate(names)}
    ptr.update(over)
    return [ptr[n] for n in names]


def conv(B=2, T=5, C=16, W=4, dtype=1, act=1, sb=80, st=16, null=False, **over):
    p = mixer.ConvProblem(B, T, C, W, dtype, act, sb, st)
    return native.lib().gdn_conv_fwd(None if null else ctypes.byref(p), *pointers(CONV_ARGS, over), None)


def scan(B=2, T=5, D=16, N=16, G=1, dtype=1, flags=1, reserved=0, strides=None, ws=1 << 32, null=False,
         **over):
    strides = strides or (T * D, D) * 3 + (T * G * N, G * N) * 2
    p = mixer.ScanProblem(B, T, D, N, G, dtype, flags, reserved, *strides)
    return native.lib().gdn_scan_fwd(None if null else ctypes.byref(p), *pointers(SCAN_ARGS, over), ws,
                                     None)


def norm(B=2, T=5, C=16, G=4, dtype=1, act=1, eps=1e-5, reserved=0, strides=None, null=False, **over):
    strides = strides or (T * C, C) * 2
    p = mixer.GroupNormProblem(B, T, C, G, dtype, act, eps, reserved, *strides)
    return native.lib().gdn_group_norm(None if null else ctypes.byref(p), *pointers(NORM_ARGS, over),
                                       None)


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(T=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(act=3), INVALID), (dict(sb=-1), INVALID), (dict(st=-1), INVALID),
    (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None), INVALID),
    (dict(x=fake(0) + 1), ALIGNMENT), (dict(lengths=fake(4) + 2), ALIGNMENT),
    (dict(weight=fake(1) + 4), ALIGNMENT), (dict(bias=fake(2) + 8), ALIGNMENT),
    (dict(state_in=fake(3) + 2), ALIGNMENT), (dict(y=fake(5) + 8), ALIGNMENT),
    (dict(state_out=fake(6) + 4), ALIGNMENT),
    # overlaps: y over x, over the state; the states shifted against each other
    (dict(y=fake(0)), INVALID), (dict(y=fake(0) + 2 * 5 * 16 * 2 - 16), INVALID),
    (dict(y=fake(3)), INVALID), (dict(y=fake(6)), INVALID), (dict(state_out=fake(3) + 16), INVALID),
    (dict(state_out=fake(1)), INVALID), (dict(state_out=fake(0)), INVALID),
])
def test_conv_refusals(kw, status):
    assert conv(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(N=0), INVALID),
    (dict(G=0), INVALID), (dict(T=-1), INVALID), (dict(D=18, G=4), INVALID), (dict(dtype=-1), INVALID),
    (dict(flags=2), INVALID), (dict(reserved=1), INVALID),
    (dict(strides=(-1,) + (80,) * 9), INVALID), (dict(strides=(80,) * 9 + (-1,)), INVALID),
    (dict(N=129), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("x", "dt", "A", "Bm", "Cm", "y")],
    *[({n: fake(SCAN_ARGS.index(n)) + 1}, ALIGNMENT) for n in ("x", "dt", "z", "Bm", "Cm", "lengths")],
    *[({n: fake(SCAN_ARGS.index(n)) + 8}, ALIGNMENT) for n in ("A", "skip", "dt_bias", "h0", "y",
                                                              "h_final", "workspace")],
    *[(dict(y=fake(SCAN_ARGS.index(n))), INVALID) for n in SCAN_ARGS if n not in ("y", "workspace")],
    (dict(h_final=fake(8) + 64), INVALID), (dict(h_final=fake(2)), INVALID),
])
def test_scan_refusals(kw, status):
    assert scan(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(G=0), INVALID),
    (dict(C=18), INVALID), (dict(T=-1), INVALID), (dict(dtype=3), INVALID), (dict(act=-1), INVALID),
    (dict(eps=-1e-5), INVALID), (dict(eps=float("nan")), INVALID), (dict(reserved=1), INVALID),
    (dict(strides=(-1, 16, 80, 16)), INVALID), (dict(strides=(80, 16, 80, -1)), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID),
    *[({n: fake(NORM_ARGS.index(n)) + 1}, ALIGNMENT) for n in ("x", "gate", "lengths")],
    *[({n: fake(NORM_ARGS.index(n)) + 8}, ALIGNMENT) for n in ("weight", "bias", "y")],
    # in place only with x contiguous and the same rows
    (dict(y=fake(0), strides=(160, 32, 80, 16)), INVALID), (dict(y=fake(0) + 16), INVALID),
    (dict(y=fake(3)), INVALID), (dict(y=fake(1)), INVALID),
])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status


def test_scan_workspace():
    for B, T, D, N in ((1, 1, 2048, 16), (256, 1, 4096, 16), (64, 4096, 4096, 16)):
        assert gdn.scan_workspace_bytes(B, T, D, N) == 0
    with pytest.raises(gdn.GdnError) as e:
        gdn.scan_workspace_bytes(1, 16, 8, 129)
    assert e.value.status == UNSUPPORTED
    with pytest.raises(gdn.GdnError) as e:
        gdn.scan_workspace_bytes(1, 16, 9, 16, 2)
    assert e.value.status == INVALID


def test_scan_needs_its_workspace():
    """One long sequence of few channels is cut into segments."""
    need = gdn.scan_workspace_bytes(1, 4096, 64, 16)
    assert need > 0
    kw = dict(B=1, T=4096, D=64)
    assert scan(**kw, ws=need - 1) == WORKSPACE
    assert scan(**kw, workspace=None) == WORKSPACE
    assert scan(**kw, workspace=fake(12) + 8) == ALIGNMENT
    for n in ("x", "y", "h_final", "h0"):
        assert scan(**kw, workspace=fake(SCAN_ARGS.index(n))) == INVALID


@pytest.mark.parametrize("call,kw", [(conv, dict(C=1 << 20, T=1 << 12)), (scan, dict(D=(1 << 24) + 16)),
                                     (norm, dict(B=(1 << 26) + 1)), (norm, dict(C=65536, G=65536)),
                                     # one token or channel with 32-bit indexes at their end
                                     (conv, dict(C=(1 << 31) - 1, T=1)), (conv, dict(C=1, T=(1 << 31) - 1)),
                                     (conv, dict(C=(1 << 31) - 1, T=0)), (conv, dict(C=(1 << 15) + 1, T=1 << 15)),
                                     (scan, dict(D=1, N=1, T=(1 << 31) - 1)),
                                     (norm, dict(C=(1 << 31) - 1, G=1, T=1)),
                                     (norm, dict(C=1, G=1, T=(1 << 31) - 1))])
def test_sizes_beyond_the_grids(call, kw):
    assert call(**kw) == UNSUPPORTED


def test_wrappers_take_cuda_tensors_only():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        gdn.conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError):
        gdn.scan_fwd(x, x, torch.zeros(8, 4), x[..., None, :4], x[..., None, :4])
    with pytest.raises(ValueError):
        gdn.group_norm(x, 2)
