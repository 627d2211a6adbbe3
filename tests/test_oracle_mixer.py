"""Facts that pin the fp64 forms of the convolution, the scan and the group norm."""
import numpy as np
import pytest

from oracle import mixer, recurrence


def test_conv_is_the_shifted_sum_and_carries_its_window():
    r = np.random.default_rng(0)
    x, w, st = r.normal(size=(2, 9, 5)), r.normal(size=(5, 4)), r.normal(size=(2, 3, 5))
    y, out, _, _ = mixer.conv(x, w, state=st, act_name="none")
    for c in range(5):
        full = np.convolve(np.concatenate([st[1, :, c], x[1, :, c]]), w[c, ::-1], "valid")
        assert np.allclose(full, y[1, :, c], atol=1e-14)
    assert (out == x[:, -3:]).all()
    y1, s1, _, _ = mixer.conv(x[:, :2], w, state=st, act_name="none")
    y2, s2, _, _ = mixer.conv(x[:, 2:], w, state=s1, act_name="none")
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(s2, out)


def test_scan_closed_form_and_split():
    r = np.random.default_rng(1)
    B, T, D, N = 2, 6, 4, 3
    x, dt = r.normal(size=(B, T, D)), r.uniform(0.1, 1, size=(B, T, D))
    A, bm, cm = -r.uniform(0.5, 2, size=(D, N)), r.normal(size=(B, T, 2, N)), r.normal(size=(B, T, 2, N))
    h0 = r.normal(size=(B, D, N))
    y, h, _, _ = mixer.scan(x, dt, A, bm, cm, h0=h0)
    for b in range(B):
        for d in range(D):
            g = d // 2
            want = sum(cm[b, -1, g] * np.exp(A[d] * dt[b, s + 1:, d].sum()) * dt[b, s, d] * x[b, s, d]
                       * bm[b, s, g] for s in range(T))
            want = want + cm[b, -1, g] * np.exp(A[d] * dt[b, :, d].sum()) * h0[b, d]
            assert np.isclose(want.sum(), y[b, -1, d], atol=1e-12)
    y1, h1, _, _ = mixer.scan(x[:, :4], dt[:, :4], A, bm[:, :4], cm[:, :4], h0=h0)
    y2, h2, _, _ = mixer.scan(x[:, 4:], dt[:, 4:], A, bm[:, 4:], cm[:, 4:], h0=h1)
    assert np.allclose(np.concatenate([y1, y2], 1), y, atol=1e-14) and np.allclose(h2, h, atol=1e-14)


def test_scan_is_the_rule_without_its_delta_term():
    """With A = -1 for every state, beta = 1 and k = B one-hot on a fresh state, S^T q of the
    gated rule and C.h of the scan agree: both add one outer product per token."""
    r = np.random.default_rng(2)
    T, N, P = 4, 4, 3
    gamma = -r.uniform(0.1, 1, size=T)
    v, q = r.normal(size=(1, T, 1, P)), r.normal(size=(1, T, 1, N))
    k = np.eye(N)[None, :, None, :]
    o, _ = recurrence.forward(q, k, v, gamma[None, :, None], np.ones((1, T, 1)), 1.0, None, chunk=1)
    dt = np.repeat(-gamma[None, :, None], P, axis=2)
    y, _, _, _ = mixer.scan(v[:, :, 0] / dt, dt, -np.ones((P, N)), k, q)
    assert np.allclose(o[:, :, 0], y, atol=1e-12)


def test_group_norm_moments_and_lengths():
    r = np.random.default_rng(3)
    x = r.normal(size=(2, 7, 12)) * 3 + 5
    y, _, _, _ = mixer.group_norm(x, 3, eps=0.0, lengths=[7, 4])
    for b, n in ((0, 7), (1, 4)):
        g = y[b, :n].reshape(n, 3, 4)
        assert np.allclose(g.mean((0, 2)), 0, atol=1e-12) and np.allclose(g.var((0, 2)), 1, atol=1e-12)
    assert np.isnan(y[1, 4:]).all()


@pytest.mark.parametrize("name", ["none", "silu", "sigmoid"])
def test_activations(name):
    v = np.array([-800.0, -1.0, 0.0, 2.0, 800.0])
    s = np.array([0.0, 1 / (1 + np.e), 0.5, 1 / (1 + np.exp(-2.0)), 1.0])
    assert np.allclose(mixer.act(v, name), {"none": v, "silu": v * s, "sigmoid": s}[name])
