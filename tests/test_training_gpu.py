"""The gated linear recurrence, layer norm and the gradients on the GPU against their
fp64 forms, elementwise within the bounds that those forms carry."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import native, training
from oracle import mixer as mixer_ref
from oracle import training as ref
from tests.mixer_bounds import check, untouched
from tests.test_mixer_gpu import FILL, draw, f64, gen, ragged, spoil

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def lengths_of(n):
    return None if n is None else n.tolist()


def checked(got, want, bound, types):
    """Every value of `want` that is not None against the bound, in its type."""
    for name, w in want.items():
        if w is None:
            assert got[name] is None, name
        else:
            check(got[name], w, bound[name], types.get(name, F32), name)


def filled(shape, dtype):
    return torch.full(shape, FILL, dtype=dtype, device="cuda")


# -------------------------------------------------------- gated linear recurrence
def recur_inputs(B, T, D, dtype, seed, rate=True, gate=True, scaling="root", state=True, strided=False,
                 lengths=False, spread=1.0):
    g = gen(seed)
    x, decay = draw(g, (B, T, D), dtype, strided), draw(g, (B, T, D), dtype, strided)
    decay.mul_(spread)
    r = (8 * torch.rand(D, generator=g) ** 3 + 0.002).cuda() if rate else None
    gt = draw(g, (B, T, D), dtype, strided) if gate else None
    h0 = torch.randn(B, D, generator=g).cuda() if state else None
    n = ragged(B, T, seed) if lengths else None
    i = dict(x=x, decay=decay, rate=r, gate=gt, scaling=scaling, h0=h0, lengths=n)
    if lengths:
        for name in ("x", "decay", "gate"):
            if i[name] is not None:
                spoil(i[name], n)
    return i


def recur_ref(i):
    return ref.recur(f64(i["x"]), f64(i["decay"]), f64(i["rate"]), f64(i["gate"]), i["scaling"], f64(i["h0"]),
                     lengths_of(i["lengths"]), gdn.RECUR_EVERY)


def recur_bwd_ref(dy, i, dh):
    return ref.recur_bwd(f64(dy), f64(i["x"]), f64(i["decay"]), f64(i["rate"]), f64(i["gate"]), i["scaling"],
                         f64(i["h0"]), f64(dh), lengths_of(i["lengths"]), gdn.RECUR_EVERY)


FORMS = [dict(rate=True, gate=True, scaling="root", state=False),
         dict(rate=True, gate=False, scaling="complement", lengths=True, strided=True),
         dict(rate=False, gate=True, scaling="root", lengths=True),
         dict(rate=False, gate=False, scaling="none", strided=True),
         dict(rate=True, gate=True, scaling="none", lengths=True),
         dict(rate=False, gate=True, scaling="complement", state=False)]

RECUR_SIZES = [(1, 1, 1), (3, 2, 8), (2, 17, 65), (4, 130, 264), (2, 1025, 40), (1, 64, 1003), (3, 5, 2048),
               (2, 300, 96), (1, 129, 68), (5, 16, 33), (2, 257, 30)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", RECUR_SIZES)
def test_recur(size, dtype):
    for k, form in enumerate(FORMS):
        i = recur_inputs(*size, dtype, 700 + k, **form)
        B, T, D = size
        out = filled(size, dtype)
        kept = filled((B, (T + 15) // 16, D), F32)
        y, h, states = gdn.recur_fwd(**i, output_states=True, out=out, states=kept)
        assert y is out and states is kept
        want, bound, _ = recur_ref(i)
        checked(dict(y=y, h=h, states=states), want, bound, dict(y=dtype))
        untouched(y, want["y"], FILL)
        untouched(states, want["states"], FILL)
        again, h2 = gdn.recur_fwd(**i, output_final_state=False)
        assert h2 is None
        at = ~np.isnan(want["y"])
        assert (f64(again)[at] == f64(y)[at]).all() and (f64(again)[~at] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", RECUR_SIZES)
def test_recur_bwd(size, dtype):
    for k, form in enumerate(FORMS):
        i = recur_inputs(*size, dtype, 720 + k, **form)
        g = gen(740 + k)
        dy = draw(g, size, dtype, form.get("strided", False))
        if i["lengths"] is not None:
            spoil(dy, i["lengths"])
        dh = torch.randn(size[0], size[2], generator=g).cuda() if k % 2 else None
        _, _, states = gdn.recur_fwd(**i, output_states=True)
        if i["lengths"] is not None:         # of chunks behind a sequence none is read
            nan = np.isnan(recur_ref(i)[0]["states"])
            states[torch.from_numpy(nan).cuda()] = float("nan")
        h0 = i.pop("h0")
        outs = dict(dx=filled(size, dtype), d_decay=filled(size, dtype),
                    d_gate=filled(size, dtype) if form["gate"] else None)
        got = gdn.recur_bwd(dy, states=states, d_final_state=dh, **i, **outs)
        i["h0"] = h0
        want, bound = recur_bwd_ref(dy, i, dh)
        names = ("dx", "d_decay", "d_gate", "d_rate", "d_state")
        checked(dict(zip(names, got)), want, bound, dict(dx=dtype, d_decay=dtype, d_gate=dtype))
        for name in ("dx", "d_decay", "d_gate"):
            if outs[name] is not None:
                untouched(outs[name], want[name], FILL)
        # outputs of its own, the last state's gradient in place
        i.pop("h0")
        d = None if dh is None else dh.clone()
        more = gdn.recur_bwd(dy, states=states, d_final_state=d, **i, d_state=d)
        assert d is None or more[4] is d
        for a, b in zip(more, got):
            if a is not None:
                live = slice(None) if a.dim() < 3 else ~torch.from_numpy(np.isnan(want["dx"])).cuda()
                assert torch.equal(a[live], b[live])
                if a.dim() == 3:
                    assert (a[~live] == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(1, 4001, 16), (2, 3000, 24), (1, 2050, 8), (3, 700, 40), (1, 6000, 130)])
def test_recur_long_sequences_of_few_channels(size, dtype):
    for k, form in enumerate((FORMS[0], FORMS[2])):
        i = recur_inputs(*size, dtype, 760 + k, **form)
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        want, bound, _ = recur_ref(i)
        checked(dict(y=y, h=h, states=states), want, bound, dict(y=dtype))
        dy = draw(gen(770), size, dtype)
        h0 = i.pop("h0")
        got = gdn.recur_bwd(dy, states=states, **i)
        i["h0"] = h0
        want, bound = recur_bwd_ref(dy, i, None)
        checked(dict(zip(("dx", "d_decay", "d_gate", "d_rate", "d_state"), got)), want, bound,
                dict(dx=dtype, d_decay=dtype, d_gate=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recur_steps_continue_a_prompt(dtype):
    i = recur_inputs(5, 40, 72, dtype, 780)
    want, bound, _ = recur_ref(i)
    cut = lambda a, b: {k: v[:, a:b] if k in ("x", "decay", "gate") else v for k, v in i.items()
                        if k not in ("h0", "lengths")}
    y0, state = gdn.recur_fwd(**cut(0, 33), h0=i["h0"])
    ys = [y0]
    for a, b in ((33, 34), (34, 35), (35, 38), (38, 40)):
        y, s = gdn.recur_step(**cut(a, b), state=state)
        assert s is state
        ys.append(y)
    checked(dict(y=torch.cat(ys, 1), h=state), dict(y=want["y"], h=want["h"]), bound, dict(y=dtype))
    whole = i["h0"].clone()
    y, h = gdn.recur_fwd(**{**i, "h0": whole}, final_state=whole)
    assert h is whole
    checked(dict(y=y, h=h), dict(y=want["y"], h=want["h"]), bound, dict(y=dtype))
    apart = torch.empty_like(state)
    y, s = gdn.recur_step(**cut(0, 1), state=i["h0"], state_out=apart)
    assert s is apart


@pytest.mark.parametrize("B,T,D", [(1, 1, 2048), (256, 1, 520), (300, 3, 64), (7, 4, 1003), (70, 2, 4096)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recur_few_tokens(dtype, B, T, D):
    for k, form in enumerate(FORMS[:4]):
        i = recur_inputs(B, T, D, dtype, 790 + k, **form)
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        want, bound, _ = recur_ref(i)
        checked(dict(y=y, h=h, states=states), want, bound, dict(y=dtype))


@pytest.mark.parametrize("scaling", ["root", "complement", "none"])
@pytest.mark.parametrize("rate", [True, False])
def test_recur_extreme_gates(rate, scaling):
    """Gates far on either side: factors of 0 and 1, no input, no gradient, no NaN."""
    B, T, D = 2, 70, 40
    i = recur_inputs(B, T, D, F32, 800, rate=rate, scaling=scaling)
    far = torch.tensor([0.0, 20.0, -20.0, 60.0, -60.0, 150.0, -150.0, float("inf"), -float("inf")])
    g = gen(801)
    for name in ("decay", "gate"):
        at = torch.randint(0, len(far), (B, T, D), generator=g)
        i[name] = far[at].cuda()
    if rate:
        i["rate"][::5] = 300.0
    y, h, states = gdn.recur_fwd(**i, output_states=True)
    want, bound, _ = recur_ref(i)
    checked(dict(y=y, h=h, states=states), want, bound, {})
    dy, dh = draw(g, (B, T, D), F32), torch.randn(B, D, generator=g).cuda()
    h0 = i.pop("h0")
    got = gdn.recur_bwd(dy, states=states, d_final_state=dh, **i)
    i["h0"] = h0
    want, bound = recur_bwd_ref(dy, i, dh)
    checked(dict(zip(("dx", "d_decay", "d_gate", "d_rate", "d_state"), got)), want, bound, {})


@pytest.mark.parametrize("scaling", ["root", "complement"])
@pytest.mark.parametrize("rate", [True, False])
def test_recur_where_factors_leave_the_normal_range(rate, scaling):
    """sigmoid(decay) and 1 - a on both sides of 2^-126, down to where they vanish."""
    i = recur_inputs(2, 50, 64, F32, 805, rate=rate, scaling=scaling)
    i["decay"] = (84 + 6 * torch.rand(2, 50, 64, generator=gen(806))).cuda() * (-1 if rate else 1)
    y, h, states = gdn.recur_fwd(**i, output_states=True)
    want, bound, _ = recur_ref(i)
    checked(dict(y=y, h=h, states=states), want, bound, {})
    dy = draw(gen(807), (2, 50, 64), F32)
    h0 = i.pop("h0")
    got = gdn.recur_bwd(dy, states=states, **i)
    i["h0"] = h0
    want, bound = recur_bwd_ref(dy, i, None)
    checked(dict(zip(("dx", "d_decay", "d_gate", "d_rate", "d_state"), got)), want, bound, {})


def test_recur_keeps_a_state_that_no_token_changes():
    """decay far below 0: a = 1 exactly, no input, so the state and its gradient pass whole.
    The sigmoid may be 2^-126 for 0; with rates up to 8, m is then 2^-61 at most, as is rate s
    / m, and x and the gradients are below 8: the others within 2^-55, d_rate, a sum of up
    to 2048 of them over rates of 0.002 at least, 2^9 m, within 2^-35."""
    for T in (1, 7, 130, 1024):
        i = recur_inputs(2, T, 40, F32, 810)
        i["decay"].fill_(-float("inf"))
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        assert torch.equal(h, i["h0"]) and torch.equal(y, h[:, None].expand_as(y))
        dh = torch.randn(2, 40, generator=gen(811)).cuda()
        h0 = i.pop("h0")
        dx, dd, dg, dr, d0 = gdn.recur_bwd(torch.zeros_like(y), states=states, d_final_state=dh, **i)
        assert torch.equal(d0, dh)
        for v, bound in ((dx, 2.0 ** -55), (dd, 2.0 ** -55), (dg, 2.0 ** -55), (dr, 2.0 ** -35)):
            assert abs(v).max() <= bound


def test_recur_empty():
    x = torch.empty(2, 0, 8, device="cuda")
    h0, rate = torch.randn(2, 8, device="cuda"), torch.rand(8, device="cuda")
    y, h, states = gdn.recur_fwd(x, x, rate, x, h0=h0, output_states=True)
    assert y.shape == (2, 0, 8) and torch.equal(h, h0) and states.shape == (2, 0, 8)
    assert (gdn.recur_fwd(x, x)[1] == 0).all()
    dx, dd, dg, dr, d0 = gdn.recur_bwd(x, x, x, states, rate, x, d_final_state=h0)
    assert dx.shape == x.shape and (dr == 0).all() and torch.equal(d0, h0)
    assert (gdn.recur_bwd(x, x, x, states)[4] == 0).all()


# -------------------------------------------------------------------- layer norm
NORM_SIZES = [(1, 1, 1), (2, 3, 8), (3, 17, 65), (1, 5, 2048), (2, 300, 96), (1, 40, 1003), (4, 2, 4096),
              (1, 3, 5000), (1, 2, 16384), (2, 7, 12289), (1, 1200, 40), (1, 2, 40000), (1, 3, 20001)]


def norm_inputs(B, T, C, dtype, seed, affine=True, strided=False, lengths=False, offset=1.0):
    g = gen(seed)
    x = draw(g, (B, T, C), dtype, strided)
    x.mul_(0.5 + torch.rand(C, generator=g).cuda()).add_(offset * torch.randn(C, generator=g).cuda())
    w = (1 + 0.3 * torch.randn(C, generator=g)).cuda() if affine else None
    b = torch.randn(C, generator=g).cuda() if affine else None
    dy = draw(g, (B, T, C), dtype, strided)
    n = ragged(B, T, seed) if lengths else None
    if lengths:
        spoil(x, n)
        spoil(dy, n)
    return x, w, b, dy, n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", NORM_SIZES)
def test_layer_norm(size, dtype):
    for k, (affine, center, strided, lengths) in enumerate(((True, True, False, False), (True, False, True, True),
                                                            (False, True, True, True), (True, True, True, False))):
        x, w, b, dy, n = norm_inputs(*size, dtype, 820 + k, affine, strided, lengths)
        if k == 3:
            b = None
        out, kept = filled(size, dtype), filled((*size[:2], 2), F32)
        y, stats = gdn.layer_norm(x, w, b, center=center, lengths=n, output_stats=True, out=out, stats=kept)
        want, bound = ref.layer_norm(f64(x), f64(w), f64(b), 1e-5, center, lengths_of(n))
        checked(dict(y=y, stats=stats), want, bound, dict(y=dtype))
        untouched(y, want["y"], FILL)
        untouched(stats, want["stats"], FILL)
        assert torch.equal(gdn.layer_norm(x, w, b, center=center, lengths=n, out=filled(size, dtype)), y)
        outs = dict(dx=filled(size, dtype))
        dx, dw, db = gdn.layer_norm_bwd(dy, x, stats, w, bias=b is not None, center=center, lengths=n, **outs)
        want, bound = ref.layer_norm_bwd(f64(dy), f64(x), f64(w), 1e-5, center, lengths_of(n))
        if w is None:
            want["d_weight"] = None
        if b is None:
            want["d_bias"] = None
        checked(dict(dx=dx, d_weight=dw, d_bias=db), want, bound, dict(dx=dtype))
        untouched(dx, want["dx"], FILL)
        again = gdn.layer_norm_bwd(dy, x, stats, w, bias=b is not None, center=center, lengths=n)
        live = ~torch.from_numpy(np.isnan(want["dx"])).cuda()
        assert torch.equal(again[0][live], dx[live]) and (again[0][~live] == 0).all()
        assert (dw is None or torch.equal(again[1], dw)) and (db is None or torch.equal(again[2], db))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_norm_of_far_and_of_constant_rows(dtype):
    """A mean of a hundred deviations; rows of one value (their deviation is eps's)."""
    x, w, b, dy, _ = norm_inputs(2, 9, 264, dtype, 830, offset=0.0)
    x += 100
    x[:, ::2] = 3.0
    y, stats = gdn.layer_norm(x, w, b, output_stats=True)
    want, bound = ref.layer_norm(f64(x), f64(w), f64(b))
    checked(dict(y=y, stats=stats), want, bound, dict(y=dtype))
    dx, dw, db = gdn.layer_norm_bwd(dy, x, stats, w, bias=True)
    want, bound = ref.layer_norm_bwd(f64(dy), f64(x), f64(w))
    checked(dict(dx=dx, d_weight=dw, d_bias=db), want, bound, dict(dx=dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_norm_in_place(dtype):
    for C in (72, 1003, 9000, 40000):
        x, w, b, _, _ = norm_inputs(2, 5, C, dtype, 840)
        want = gdn.layer_norm(x, w, b)
        assert gdn.layer_norm(x, w, b, out=x) is x and torch.equal(x, want)


@pytest.mark.parametrize("rows,C", [(3000, 64), (5001, 24), (2500, 520), (1300, 2056)])
def test_layer_norm_sums_over_many_tokens(rows, C):
    for dtype in (F32, BF16):
        x, w, b, dy, _ = norm_inputs(1, rows, C, dtype, 850)
        _, stats = gdn.layer_norm(x, w, b, output_stats=True)
        dx, dw, db = gdn.layer_norm_bwd(dy, x, stats, w, bias=True)
        want, bound = ref.layer_norm_bwd(f64(dy), f64(x), f64(w))
        checked(dict(dx=dx, d_weight=dw, d_bias=db), want, bound, dict(dx=dtype))


def test_layer_norm_empty():
    x = torch.empty(2, 0, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    y, stats = gdn.layer_norm(x, w, output_stats=True)
    dx, dw, db = gdn.layer_norm_bwd(x, x, stats, w, bias=True)
    assert y.shape == dx.shape == x.shape and (dw == 0).all() and (db == 0).all()
    x = torch.randn(2, 3, 8, device="cuda")
    none = torch.zeros(2, dtype=torch.int32, device="cuda")
    _, stats = gdn.layer_norm(x, w, output_stats=True)
    dx, dw, db = gdn.layer_norm_bwd(x, x, stats, w, bias=True, lengths=none)
    assert (dx == 0).all() and (dw == 0).all() and (db == 0).all()


# ------------------------------------------------------------- short convolution
CONV_SIZES = [(1, 1, 1), (3, 2, 8), (2, 17, 65), (4, 130, 264), (2, 1025, 40), (1, 64, 1003), (3, 3, 2048),
              (1, 3000, 24), (70, 5, 72)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("size", CONV_SIZES)
def test_conv_bwd(size, W, dtype):
    B, T, C = size
    act = ["silu", "none", "sigmoid"][(T + W) % 3]
    for k, (strided, lengths, state, bias) in enumerate(((False, False, False, False), (True, True, True, True),
                                                         (False, True, True, False), (True, False, False, True))):
        g = gen(860 + 10 * W + k)
        x, dy = draw(g, size, dtype, strided), draw(g, size, dtype, strided)
        w = (torch.randn(C, W, generator=g) * 0.5).cuda()
        b = (0.1 * torch.randn(C, generator=g)).cuda() if bias else None
        st = draw(g, (B, W - 1, C), dtype) if state else None
        dlast = draw(g, (B, W - 1, C), dtype) if k % 2 else None
        n = ragged(B, T, 870 + k) if lengths else None
        if lengths:
            spoil(x, n)
            spoil(dy, n)
        out = filled(size, dtype)
        dx, dw, db, ds = gdn.conv_bwd(dy, x, w, b, st, act, dlast, n, dx=out)
        want, bound = ref.conv_bwd(f64(dy), f64(x), f64(w), f64(b), f64(st), act, f64(dlast), lengths_of(n))
        if b is None:
            want["d_bias"] = None
        if st is None:
            want["d_state"] = None
        checked(dict(dx=dx, d_weight=dw, d_bias=db, d_state=ds), want, bound, dict(dx=dtype, d_state=dtype))
        untouched(dx, want["dx"], FILL)
        again = gdn.conv_bwd(dy, x, w, b, st, act, dlast, n)       # outputs of its own
        live = ~torch.from_numpy(np.isnan(want["dx"])).cuda()
        assert torch.equal(again[0][live], dx[live]) and (again[0][~live] == 0).all()
        for a, c in zip(again[1:], (dw, db, ds)):
            assert (a is None and c is None) or torch.equal(a, c)


def test_conv_bwd_empty():
    x = torch.empty(2, 0, 8, device="cuda")
    w, st = torch.ones(8, 4, device="cuda"), torch.randn(2, 3, 8, device="cuda")
    dx, dw, db, ds = gdn.conv_bwd(x, x, w, torch.ones(8, device="cuda"), st, d_final_state=st)
    assert dx.shape == x.shape and (dw == 0).all() and (db == 0).all() and torch.equal(ds, st)
    assert (gdn.conv_bwd(x, x, w, None, st)[3] == 0).all()
