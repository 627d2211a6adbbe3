"""Gradients at the edges of their ranges on the GPU against their fp64 forms: values that are not
finite, rates of 0, every form of the recurrence's gates, sums of very many terms."""
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from oracle import training as ref
from tests.mixer_bounds import check
from tests.test_mixer_gpu import draw, f64, gen
from tests.test_training_gpu import checked, recur_bwd_ref, recur_inputs, recur_ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GRADIENTS = ("dx", "d_decay", "d_gate", "d_rate", "d_state")


# ------------------------------------------------------------------- NaN goes on
def is_nan_in(t, at):
    """NaN exactly where `at` says so."""
    return torch.equal(torch.isnan(t), at)


@pytest.mark.parametrize("act", ["sigmoid", "silu", "none"])
@pytest.mark.parametrize("C", [72, 65])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_bwd_gives_nan_on(dtype, C, act):
    """A value before the activation that is NaN makes NaN of the gradients it enters, as the forward
    pass does of its output; without an activation no gradient but the weights' reads the input."""
    B, T, W, b, t, c = 2, 40, 4, 1, 17, 5
    g = gen(1000)
    x, dy, state = draw(g, (B, T, C), dtype), draw(g, (B, T, C), dtype), draw(g, (B, W - 1, C), dtype)
    weight, bias = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    clean = gdn.conv_bwd(dy, x, weight, bias, state, act)
    through = act != "none"

    def gradients(**changed):
        got = gdn.conv_bwd(dy, **{**dict(x=x, weight=weight, bias=bias, state=state, act=act), **changed})
        y = gdn.conv_fwd(changed.get("x", x), changed.get("weight", weight), changed.get("bias", bias), state,
                         act=act)[0]
        return got, torch.isnan(y)

    def only(got, *at):
        for v, want, where in zip(got, clean, at):
            assert is_nan_in(v, where)
            assert torch.equal(v[~where], want[~where])

    nowhere = [torch.zeros_like(v, dtype=torch.bool) for v in clean]
    # an input: the values before the activation of W tokens, the gradients of W - 1 more before them
    bad = x.clone()
    bad[b, t, c] = float("nan")
    got, y = gradients(x=bad)
    dx, dw, db, ds = (v.clone() for v in nowhere)
    assert y.any() and y[b, t:t + W, c].all()
    dx[b, t - W + 1:t + W, c] = through
    dw[c] = True
    db[c] = through
    only(got, dx, dw, db, ds)
    # a weight: every value of its channel
    bad = weight.clone()
    bad[c, 2] = float("nan")
    got, y = gradients(weight=bad)
    assert y[..., c].all()
    if through:
        dx, dw, db, ds = (v.clone() for v in nowhere)
        dx[..., c] = dw[c] = db[c] = ds[..., c] = True
        only(got, dx, dw, db, ds)
    # a bias
    bad = bias.clone()
    bad[c] = float("nan")
    got, y = gradients(bias=bad)
    dx, dw, db, ds = (v.clone() for v in nowhere)
    assert y[..., c].all()
    dx[..., c] = dw[c] = db[c] = ds[..., c] = through
    only(got, dx, dw, db, ds)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_bwd_of_far_values(dtype):
    """The sigmoid's slope where exp(-v) leaves fp32's range on either side, infinite values among
    them: 0 but for what lies below the normal range."""
    B, T, C, W = 1, 24, 16, 2
    x = torch.zeros(B, T, C, device="cuda", dtype=dtype)
    far = torch.tensor([60.0, -60.0, 87.0, -87.0, 88.0, -88.0, 126.0, -126.0, 200.0, -200.0, 1e30, -1e30, 3e38,
                        -3e38, float("inf"), -float("inf")], device="cuda")
    dy = draw(gen(1010), (B, T, C), dtype)
    dx, dw, db = gdn.conv_bwd(dy, x, torch.ones(C, W, device="cuda"), far, act="sigmoid")[:3]
    p = dy.double() * torch.exp(-far.abs().double())           # s (1 - s), whose larger factor is 1 but for 2^-86
    # a sigmoid and its complement are off by 19 + 6 |v| roundings, products and 24 additions by fewer
    # than 40; exp(-88) is below the normal range, where each factor is off by tiny
    bound = (19 + 6 * 88 + 40) * ref.U * p.abs() + 2 * ref.TINY * dy.double().abs()
    two = lambda v: torch.cat([v[:, :-1] + v[:, 1:], v[:, -1:]], 1)
    check(dx, f64(two(p)), f64(two(bound)), dtype)
    check(db, f64(p.sum((0, 1))), f64(bound.sum((0, 1))), F32)
    assert (dw == 0).all()


# ---------------------------------------------------------------------- rates of 0
@pytest.mark.parametrize("scaling", ["root", "complement", "none"])
@pytest.mark.parametrize("size", [(2, 5, 72), (2, 50, 72), (3, 150, 65), (1, 2100, 16)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recur_channels_of_rate_zero(dtype, size, scaling):
    """A channel whose rate is 0 keeps its state whole; the root's factor m is 0 there and its
    gradient counts as 0, in the rate's gradient too."""
    B, T, D = size
    for gate in (True, False):
        i = recur_inputs(*size, dtype, 1100, gate=gate, scaling=scaling, lengths=B > 1)
        i["rate"][::3] = 0.0
        i["rate"][1::6] = -0.0
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        want, bound, _ = recur_ref(i)
        checked(dict(y=y, h=h, states=states), want, bound, dict(y=dtype))
        dy, dh = draw(gen(1101), size, dtype), torch.randn(B, D, generator=gen(1102)).cuda()
        h0 = i.pop("h0")
        got = gdn.recur_bwd(dy, states=states, d_final_state=dh, **i)
        i["h0"] = h0
        want, bound = recur_bwd_ref(dy, i, dh)
        if scaling == "root":
            # m's gradient is 0, so the rate's is -sum lam s a h: no larger than its terms
            size_of = abs(want["d_rate"][::3]).max()
            assert size_of < 1e6 and abs(got[3][::3]).max() < 2 * size_of
        checked(dict(zip(GRADIENTS, got)), want, bound, dict(dx=dtype, d_decay=dtype, d_gate=dtype))


def test_recur_rates_below_the_normal_range():
    """They count as 0 for m, as 1 - a^2 does in the forward pass: the state passes whole, x adds
    nothing to it, and the rate's gradient is that of the decay alone."""
    B, T, D = 2, 50, 40
    i = recur_inputs(B, T, D, F32, 1110)
    i["rate"].copy_(torch.tensor([1e-38, 1e-39, 1e-40, 1e-44, 0.0])[torch.arange(D) % 5])
    y, h, states = gdn.recur_fwd(**i, output_states=True)
    assert torch.equal(h, i["h0"]) and torch.equal(y, h[:, None].expand_as(y))
    dy = draw(gen(1111), (B, T, D), F32)
    h0 = i.pop("h0")
    dx, dd, dg, dr, d0 = gdn.recur_bwd(dy, states=states, **i)
    lam = dy.double().flip(1).cumsum(1).flip(1)
    s = torch.sigmoid(i["decay"].double())
    terms = -lam * s * h0.double()[:, None]
    # lam is off by 60 roundings of its terms, the sigmoid by 7 + 2 |v|, |v| < 6; 100 additions, 2 products
    size = 60 * ref.U * dy.double().abs().sum(1, keepdim=True) * s * h0.double().abs()[:, None] \
        + (7 + 12 + 102) * ref.U * terms.abs()
    check(dr, f64(terms.sum((0, 1))), f64(size.sum((0, 1))), F32)
    # m is below 2^-62, and its gradient times any of the rates too
    small = 2.0 ** -55
    assert abs(dx).max() < small and abs(dd).max() < small and abs(dg).max() < small


@pytest.mark.parametrize("size", [(2, 6, 24), (2, 70, 24), (2, 45, 33)])
def test_recur_the_largest_rates(size):
    """2^64: decays far below 0 on both sides of where their sigmoid counts as 0 or as 2^-126, which moves m
    by 2^-30 at most (sqrt(2^65 2^-126)) and 1 - a by 2^-62; the tokens behind a sequence pass its state whole."""
    B, T, D = size
    i = recur_inputs(*size, F32, 1120, lengths=True)
    i["rate"].fill_(2.0 ** 64)
    far = torch.tensor([-float("inf"), -200.0, -100.0, -88.0, -87.0, -80.0, -60.0, -30.0, 0.0, 90.0])
    inside = torch.isfinite(i["x"])
    decay = far[torch.randint(0, 10, size, generator=gen(1121))].cuda()
    i["decay"] = torch.where(inside, decay, torch.full_like(decay, float("nan")))
    y, h, states = gdn.recur_fwd(**i, output_states=True)
    want, bound, _ = recur_ref(i)
    off = 2.0 ** -30 * float(i["x"].nan_to_num(0.0).abs().sum(1).max())
    checked(dict(y=y, h=h, states=states), want, {k: v + off for k, v in bound.items()}, {})
    i["decay"] = torch.where(inside, torch.full_like(decay, -float("inf")), i["decay"])
    y, h, states = gdn.recur_fwd(**i, output_states=True)
    assert torch.equal(h, i["h0"])
    dy, dh = torch.zeros_like(y), torch.randn(B, D, generator=gen(1122)).cuda()
    dx, dd, dg, _, d0 = gdn.recur_bwd(dy, states=states, d_final_state=dh,
                                      **{k: v for k, v in i.items() if k != "h0"})
    assert torch.equal(d0, dh)
    for v in (dx, dd, dg):
        assert abs(v).max() <= 2.0 ** -24


# ----------------------------------------------------------------- every form of gates
@pytest.mark.parametrize("scaling", ["none", "complement", "root"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_recur_every_form(dtype, rate, gate, scaling):
    """Each form has kernels of its own: for rows of whole pieces (72), for others with an even and an odd
    number of channels, and for a few tokens."""
    for k, size in enumerate(((2, 40, 72), (2, 40, 65), (3, 37, 66), (2, 5, 72), (2, 7, 65))):
        i = recur_inputs(*size, dtype, 1200 + k, rate, gate, scaling, lengths=k % 2 == 1)
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        want, bound, _ = recur_ref(i)
        checked(dict(y=y, h=h, states=states), want, bound, dict(y=dtype))
        dy = draw(gen(1210 + k), size, dtype)
        dh = torch.randn(size[0], size[2], generator=gen(1220 + k)).cuda()
        h0 = i.pop("h0")
        got = gdn.recur_bwd(dy, states=states, d_final_state=dh, **i)
        i["h0"] = h0
        want, bound = recur_bwd_ref(dy, i, dh)
        checked(dict(zip(GRADIENTS, got)), {n: want[n] for n in GRADIENTS}, bound,
                dict(dx=dtype, d_decay=dtype, d_gate=dtype))


# -------------------------------------------------------------- sums of very many terms
def sum_is(got, terms, additions, each):
    """`terms` (fp64) summed over batch and tokens in fp32, every one of them off by `each` roundings
    and at most `additions` additions behind it."""
    total, size = terms.sum((0, 1)), terms.abs().sum((0, 1))
    check(got, f64(total), f64(size) * (additions + each) * ref.U, F32)


def test_layer_norm_sums_behind_the_bounds_of_the_form():
    """Rows that take a block: each of 304 adds up 900 of them, more than the fp64 form's bound counts."""
    rows, C = 304 * 900, 1032
    x = torch.randn(1, rows, C, device="cuda", generator=torch.Generator("cuda").manual_seed(1300))
    dy = torch.randn(1, rows, C, device="cuda", generator=torch.Generator("cuda").manual_seed(1301))
    w = torch.rand(C, generator=gen(1302)).cuda()
    _, stats = gdn.layer_norm(x, w, output_stats=True)
    _, dw, db = gdn.layer_norm_bwd(dy, x, stats, w, bias=True)
    additions = ref.additions(rows / 304, 304)
    assert additions > ref.SUMS
    xhat = x.double().sub_(stats[..., :1]).mul_(stats[..., 1:])     # two roundings in fp32
    sum_is(dw, xhat.mul_(dy), additions, 3)
    del xhat
    sum_is(db, dy.double(), additions, 0)


def test_recur_sums_behind_the_bounds_of_the_form():
    """Without clusters a lane adds up every sixth tile of 16 tokens. The terms of the rate's gradient by the
    decay's, d_decay = -dlog rate s (1 - s): the same products but for rate and 1 - s."""
    B, T, D = 2, 8192, 64 * 77
    g = torch.Generator("cuda").manual_seed(1310)
    x, decay, dy = (torch.randn(B, T, D, device="cuda", generator=g) for _ in range(3))
    rate = (0.05 + torch.rand(D, generator=gen(1311))).cuda()
    _, _, states = gdn.recur_fwd(x, decay, rate, scaling="none", output_states=True)
    d_decay, d_rate = gdn.recur_bwd(dy, x, decay, states, rate, scaling="none")[1:4:2]
    terms = d_decay.double().div_(rate).div_(torch.sigmoid(-decay.double()))
    additions = ref.additions(T / 6 + 16 + 6, B)
    assert additions > ref.SUMS
    # 1 - s off by (12 + 4 |v|) roundings, |v| < 7; its product with s and both with the rate and dlog
    sum_is(d_rate, terms, additions, 12 + 4 * 7 + 5)
