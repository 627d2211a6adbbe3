"""The fp64 gradients of oracle/training.py against central differences of the fp64
forward forms, and the forward forms against each other."""
import numpy as np
import pytest

from oracle import mixer, training as ref


def rng(seed):
    return np.random.default_rng(seed)


def by_differences(loss, v, step=1e-5):
    """The gradient of loss() with respect to the array v, changed in place."""
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        keep = v[i]
        v[i] = keep + step
        up = loss()
        v[i] = keep - step
        g[i] = (up - loss()) / (2 * step)
        v[i] = keep
    return g


def near(got, want):
    """Differences of step 1e-5 in fp64: truncation about 1e-10, rounding about 1e-11 of the loss."""
    want = np.where(np.isnan(want), 0, want)
    assert abs(got - want).max() < 1e-8 * max(1.0, abs(want).max())


@pytest.mark.parametrize("scaling", ["root", "complement", "none"])
@pytest.mark.parametrize("rated,gated", [(True, True), (False, True), (True, False)])
def test_recur_gradients(rated, gated, scaling):
    r = rng(1)
    B, T, D = 3, 5, 3
    lengths = [5, 0, 3]
    x, decay, dy = (r.standard_normal((B, T, D)) for _ in range(3))
    gate = r.standard_normal((B, T, D)) if gated else None
    rate = r.uniform(0.1, 1, D) if rated else None
    h0, dh = r.standard_normal((B, D)), r.standard_normal((B, D))

    def loss():
        out = ref.recur(x, decay, rate, gate, scaling, h0, lengths, every=2)[0]
        return np.nansum(out["y"] * dy) + (out["h"] * dh).sum()

    got, bound = ref.recur_bwd(dy, x, decay, rate, gate, scaling, h0, dh, lengths, every=2)
    for name, v in (("dx", x), ("d_decay", decay), ("d_gate", gate), ("d_rate", rate), ("d_state", h0)):
        if v is None:
            assert got[name] is None
        else:
            near(by_differences(loss, v), got[name])
            assert got[name].shape == bound[name].shape


def test_recur_states_and_closed_form():
    """With a constant factor and no scaling: h_t = a^t h0 + (1 - a^t) / (1 - a) x."""
    B, T, D = 2, 37, 3
    rate = np.array([0.1, 0.5, 3.0])
    x, h0 = np.ones((B, T, D)) * 0.25, np.full((B, D), 2.0)
    decay = np.full((B, T, D), 30.0)      # sigmoid 1
    out, _, _ = ref.recur(x, decay, rate, None, "none", h0, None)
    a = np.exp(-rate)
    n = np.arange(1, T + 1)[:, None]
    want = a ** n * 2.0 + (1 - a ** n) / (1 - a) * 0.25
    assert np.allclose(out["y"][0], want, rtol=1e-10)
    assert np.array_equal(out["states"][:, 1:], out["y"][:, 15::16][:, :2]) and np.array_equal(out["states"][:, 0], h0)


@pytest.mark.parametrize("center,affine", [(True, True), (False, True), (True, False)])
def test_layer_norm_gradients(center, affine):
    r = rng(2)
    x, dy = r.standard_normal((2, 3, 5)), r.standard_normal((2, 3, 5))
    w, bias = (r.standard_normal(5), r.standard_normal(5)) if affine else (None, None)
    lengths = [3, 1]
    loss = lambda: np.nansum(ref.layer_norm(x, w, bias, 1e-5, center, lengths)[0]["y"] * dy)
    got, _ = ref.layer_norm_bwd(dy, x, w, 1e-5, center, lengths)
    near(by_differences(loss, x), got["dx"])
    if affine:
        near(by_differences(loss, w), got["d_weight"])
        near(by_differences(loss, bias), got["d_bias"])


def test_layer_norm_is_the_group_norm_of_one_group():
    r = rng(3)
    x, w, bias = r.standard_normal((2, 3, 8)), r.standard_normal(8), r.standard_normal(8)
    y = ref.layer_norm(x, w, bias)[0]["y"]
    assert np.allclose(y.reshape(6, 1, 8), mixer.group_norm(x.reshape(6, 1, 8), 1, w, bias)[0], atol=1e-13)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none", "sigmoid"])
def test_conv_gradients(act, W):
    r = rng(4)
    B, T, C = 3, 5, 2
    lengths = [5, 0, 2]
    x, dy = r.standard_normal((B, T, C)), r.standard_normal((B, T, C))
    w, bias = r.standard_normal((C, W)), r.standard_normal(C)
    state, dlast = r.standard_normal((B, W - 1, C)), r.standard_normal((B, W - 1, C))

    def loss():
        y, last, _, _ = mixer.conv(x, w, bias, state, lengths, act)
        return np.nansum(y * dy) + (last * dlast).sum()

    got, _ = ref.conv_bwd(dy, x, w, bias, state, act, dlast, lengths)
    for name, v in (("dx", x), ("d_weight", w), ("d_bias", bias), ("d_state", state)):
        near(by_differences(loss, v), got[name])
