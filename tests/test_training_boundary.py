"""The C entries and wrappers of the gated linear recurrence, layer norm and the gradients
refuse bad calls before touching CUDA."""
import ctypes

import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import mixer, native, training
from tests.test_mixer_boundary import fake, pointers

INVALID, UNSUPPORTED = native.GDN_ERR_INVALID_ARG, native.GDN_ERR_UNSUPPORTED
ALIGNMENT, WORKSPACE = native.GDN_ERR_ALIGNMENT, native.GDN_ERR_WORKSPACE
FAR = 2 ** 32

RECUR = ("x", "decay", "gate", "rate", "h0", "lengths", "y", "h_final", "states")
RECUR_BWD = ("dy", "x", "decay", "gate", "rate", "states", "dh_final", "lengths", "dx", "d_decay", "d_gate",
             "d_rate", "dh0", "workspace")
NORM = ("x", "weight", "bias", "lengths", "y", "stats")
NORM_BWD = ("dy", "x", "stats", "weight", "lengths", "dx", "d_weight", "d_bias", "workspace")
CONV_BWD = ("dy", "x", "weight", "bias", "state_in", "d_state_out", "lengths", "dx", "d_weight", "d_bias",
            "d_state_in", "workspace")


def recur(bwd=False, B=2, T=5, D=16, dtype=1, scaling=2, reserved=0, strides=None, ws=1 << 32, null=False, **over):
    p = training.RecurProblem(B, T, D, dtype, scaling, reserved, *(strides or (80, 16) * 4))
    ref = None if null else ctypes.byref(p)
    if bwd:
        return native.lib().gdn_recur_bwd(ref, *pointers(RECUR_BWD, over), ws, None)
    return native.lib().gdn_recur_fwd(ref, *pointers(RECUR, over), None)


def norm(bwd=False, B=2, T=5, C=16, dtype=1, flags=0, eps=1e-5, strides=None, ws=1 << 32, null=False, **over):
    p = training.LayerNormProblem(B, T, C, dtype, flags, eps, *(strides or (80, 16) * 2))
    ref = None if null else ctypes.byref(p)
    if bwd:
        return native.lib().gdn_layer_norm_bwd(ref, *pointers(NORM_BWD, over), ws, None)
    return native.lib().gdn_layer_norm(ref, *pointers(NORM, over), None)


def conv(B=2, T=5, C=16, W=4, dtype=1, act=1, strides=None, ws=1 << 32, null=False, **over):
    p = training.ConvBwdProblem(B, T, C, W, dtype, act, *(strides or (80, 16) * 2))
    return native.lib().gdn_conv_bwd(None if null else ctypes.byref(p), *pointers(CONV_BWD, over), ws, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(D=0), INVALID), (dict(T=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(scaling=3), INVALID), (dict(scaling=-1), INVALID), (dict(reserved=1), INVALID),
    *[(dict(strides=(80, 16) * 4 if i < 0 else tuple(-1 if j == i else 80 for j in range(8))), INVALID)
      for i in range(8)],
    (dict(B=65536), UNSUPPORTED), (dict(D=(1 << 24) + 1), UNSUPPORTED), (dict(T=(1 << 30) + 1), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(decay=None), INVALID),
])
def test_recur_refusals(kw, status, bwd):
    assert recur(bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INVALID),
    *[({n: fake(RECUR.index(n)) + 1}, ALIGNMENT) for n in ("x", "decay", "gate")],
    (dict(lengths=fake(5) + 2), ALIGNMENT),
    *[({n: fake(RECUR.index(n)) + 8}, ALIGNMENT) for n in ("rate", "h0", "y", "h_final", "states")],
    *[(dict(y=fake(RECUR.index(n))), INVALID) for n in RECUR if n != "y"],
    *[(dict(states=fake(RECUR.index(n))), INVALID) for n in RECUR if n != "states"],
    *[(dict(h_final=fake(RECUR.index(n))), INVALID) for n in RECUR if n not in ("h_final", "h0")],
    (dict(h_final=fake(RECUR.index("h0")) + 16), INVALID),
])
def test_recur_fwd_refusals(kw, status):
    assert recur(**kw) == status


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, INVALID) for n in ("dy", "states", "dx", "d_decay", "d_gate", "gate", "rate")],
    (dict(workspace=None), WORKSPACE), (dict(ws=0), WORKSPACE),
    *[({n: fake(RECUR_BWD.index(n)) + 1}, ALIGNMENT) for n in ("dy", "x", "decay", "gate", "lengths")],
    *[({n: fake(RECUR_BWD.index(n)) + 8}, ALIGNMENT) for n in RECUR_BWD
      if n not in ("dy", "x", "decay", "gate", "lengths")],
    *[({o: fake(RECUR_BWD.index(n))}, INVALID) for o in ("dx", "d_decay", "d_gate", "d_rate", "dh0", "workspace")
      for n in RECUR_BWD if n != o and (o, n) != ("dh0", "dh_final")],
    (dict(dh0=fake(RECUR_BWD.index("dh_final")) + 16), INVALID),
])
def test_recur_bwd_refusals(kw, status):
    assert recur(True, **kw) == status


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(T=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(flags=2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    *[(dict(strides=tuple(-1 if j == i else 80 for j in range(4))), INVALID) for i in range(4)],
    (dict(C=(1 << 30) + 1), UNSUPPORTED), (dict(B=1 << 16, T=1 << 15), UNSUPPORTED),
    (dict(x=None), INVALID),
])
def test_norm_refusals(kw, status, bwd):
    assert norm(bwd, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(y=None), INVALID), (dict(x=fake(0) + 1), ALIGNMENT), (dict(lengths=fake(3) + 2), ALIGNMENT),
    *[({n: fake(NORM.index(n)) + 8}, ALIGNMENT) for n in ("weight", "bias", "y", "stats")],
    (dict(y=fake(0), strides=(160, 32, 80, 16)), INVALID), (dict(y=fake(0) + 16), INVALID),
    *[(dict(y=fake(NORM.index(n))), INVALID) for n in ("weight", "bias", "lengths", "stats")],
    *[(dict(stats=fake(NORM.index(n))), INVALID) for n in ("x", "weight", "bias", "lengths")],
])
def test_norm_fwd_refusals(kw, status):
    assert norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, INVALID) for n in ("dy", "stats", "dx")],
    (dict(workspace=None), WORKSPACE), (dict(ws=0), WORKSPACE),
    *[({n: fake(NORM_BWD.index(n)) + 1}, ALIGNMENT) for n in ("dy", "x", "lengths")],
    *[({n: fake(NORM_BWD.index(n)) + 8}, ALIGNMENT) for n in NORM_BWD if n not in ("dy", "x", "lengths")],
    *[({o: fake(NORM_BWD.index(n))}, INVALID) for o in ("dx", "d_weight", "d_bias", "workspace") for n in NORM_BWD
      if n != o],
])
def test_norm_bwd_refusals(kw, status):
    assert norm(True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(null=True), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(T=-1), INVALID),
    (dict(dtype=2), INVALID), (dict(act=3), INVALID), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED),
    *[(dict(strides=tuple(-1 if j == i else 80 for j in range(4))), INVALID) for i in range(4)],
    (dict(B=65536), UNSUPPORTED), (dict(C=1 << 20, T=1 << 12), UNSUPPORTED), (dict(C=(1 << 30) + 1, T=0), UNSUPPORTED),
    *[({n: None}, INVALID) for n in ("dy", "x", "weight", "dx", "d_weight")],
    (dict(workspace=None), WORKSPACE), (dict(ws=0), WORKSPACE),
    *[({n: fake(CONV_BWD.index(n)) + 1}, ALIGNMENT) for n in ("dy", "x", "lengths")],
    *[({n: fake(CONV_BWD.index(n)) + 8}, ALIGNMENT) for n in CONV_BWD if n not in ("dy", "x", "lengths")],
    *[({o: fake(CONV_BWD.index(n))}, INVALID) for o in ("dx", "d_weight", "d_bias", "d_state_in", "workspace")
      for n in CONV_BWD if n != o],
    (dict(d_state_in=fake(CONV_BWD.index("d_state_out")) + 16), INVALID),
])
def test_conv_bwd_refusals(kw, status):
    assert conv(**kw) == status


@pytest.mark.parametrize("call,bad", [
    (gdn.recur_bwd_workspace_bytes, [(1, 16, (1 << 24) + 1), (1, FAR + 16, 8), (FAR + 1, 16, 8), (65536, 1, 1)]),
    (gdn.layer_norm_bwd_workspace_bytes, [(1, 16, (1 << 30) + 1), (1, 16, FAR + 8), (1 << 16, 1 << 15, 8)]),
    (lambda *s: gdn.conv_bwd_workspace_bytes(*s, 4), [(1, FAR + 16, 8), (65536, 16, 8), (1, 1 << 12, 1 << 20)]),
])
def test_workspace_refusals(call, bad):
    assert call(2, 5, 16) >= 0
    for sizes in bad:
        with pytest.raises(gdn.GdnError) as e:
            call(*sizes)
        assert e.value.status == UNSUPPORTED


def test_the_kept_states_of_both_sides_agree():
    """GDN_RECUR_EVERY of the header is the wrapper's."""
    header = open(native.LIB_PATH.parents[2] / "include" / "gdn.h").read()
    assert f"GDN_RECUR_EVERY = {gdn.RECUR_EVERY} " in header


def test_wrappers_take_cuda_tensors_only():
    x, st = torch.zeros(1, 4, 8), torch.zeros(1, 1, 8)
    for call in (lambda: gdn.recur_fwd(x, x), lambda: gdn.recur_step(x, x, torch.zeros(1, 8)),
                 lambda: gdn.recur_bwd(x, x, x, st), lambda: gdn.layer_norm(x),
                 lambda: gdn.layer_norm_bwd(x, x, torch.zeros(1, 4, 2)),
                 lambda: gdn.conv_bwd(x, x, torch.zeros(8, 4))):
        with pytest.raises(ValueError):
            call()


@pytest.fixture
def anywhere(monkeypatch):
    """Plans from CPU tensors, as if these were on a device; no call follows."""
    for m in (mixer, training):
        monkeypatch.setattr(m, "_x", lambda x, axes=None: (x.shape, x.dtype, x.get_device()))


def ones(*shape):
    return torch.ones((1,) * len(shape)).expand(shape)


def test_sizes_that_32_bits_cannot_hold(anywhere):
    def refused(call):
        with pytest.raises(gdn.GdnError) as e:
            call()
        assert e.value.status == UNSUPPORTED

    for B, T, C in ((FAR + 3, 5, 1), (3, FAR + 5, 1)):
        x = ones(B, T, C)
        refused(lambda: training._recur_problem(x, x, None, None, "root", None))
        refused(lambda: training._layer_norm_problem(x, None, 1e-5, True, None))
        refused(lambda: training._conv_bwd_plan(x, x, torch.ones(1, 4), None, None, "silu", None, None, *[None] * 4))


def test_wrapper_refusals(anywhere):
    x = torch.ones(2, 5, 8)
    st = torch.ones(2, 1, 8)
    plan = lambda x=x, decay=x, rate=None, gate=None, scaling="root", h0=None, n=None, out=None, h=None, st=None: \
        training._recur_plan(x, decay, rate, gate, scaling, h0, n, out, h, st)
    assert plan()[1:] == ((2, 8), (2, 1, 8), -1)
    for kw in (dict(decay=torch.ones(2, 5, 7)), dict(rate=torch.ones(7)), dict(scaling="square"),
               dict(h0=torch.ones(2, 1, 8)), dict(st=torch.ones(2, 2, 8)), dict(n=torch.ones(3, dtype=torch.int32)),
               dict(gate=torch.ones(2, 8, 5).transpose(1, 2)), dict(out=torch.ones(2, 8, 5).transpose(1, 2))):
        with pytest.raises(ValueError):
            plan(**kw)
    for kw in (dict(decay=x.bfloat16()), dict(rate=torch.ones(8).double()), dict(h0=torch.ones(2, 8).bfloat16()),
               dict(n=torch.ones(2, dtype=torch.int64))):
        with pytest.raises(TypeError):
            plan(**kw)
    for extra in (dict(d_gate=x), dict(d_rate=torch.ones(8))):      # without a gate or a rate
        with pytest.raises(ValueError):
            training._recur_bwd_plan(x, x, x, st, None, None, "root", None, None, None, None,
                                     extra.get("d_gate"), extra.get("d_rate"), None)
    with pytest.raises(ValueError):
        training._layer_norm_bwd_plan(x, x, torch.ones(2, 5), None, True, None, None, None, None)
    with pytest.raises(ValueError):
        training._conv_bwd_plan(x, x, torch.ones(8, 4), None, torch.ones(2, 2, 8), "silu", None, None, *[None] * 4)
