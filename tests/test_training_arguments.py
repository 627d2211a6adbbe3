"""The wrappers of the recurrence's, norm's and convolution's gradients refuse a call without one of
its tensors, and buffers for gradients that the call does not have; nothing is launched."""
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import training
from tests.test_training_boundary import anywhere  # noqa: F401 (a fixture)


def x(*shape):
    return torch.ones(*shape or (2, 5, 8))


STATES, STATS, WEIGHT = x(2, 1, 8), x(2, 5, 2), x(8, 4)


@pytest.mark.parametrize("call", [
    lambda: gdn.recur_fwd(x(), None), lambda: gdn.recur_step(x(), None, x(2, 8)),
    lambda: gdn.recur_bwd(None, x(), x(), STATES), lambda: gdn.recur_bwd(x(), x(), None, STATES),
    lambda: gdn.recur_bwd(x(), x(), x(), None),
    lambda: gdn.layer_norm_bwd(None, x(), STATS), lambda: gdn.layer_norm_bwd(x(), x(), None),
    lambda: gdn.conv_bwd(None, x(), WEIGHT), lambda: gdn.conv_bwd(x(), x(), None),
])
def test_missing_tensors(anywhere, call):  # noqa: F811
    with pytest.raises(ValueError, match="must be given"):
        call()


@pytest.mark.parametrize("call", [
    lambda **k: gdn.layer_norm_bwd(x(), x(), STATS, d_weight=x(8), **k),
    lambda **k: gdn.layer_norm_bwd(x(), x(), STATS, x(8), d_bias=x(8), **k),
    lambda **k: gdn.conv_bwd(x(), x(), WEIGHT, d_bias=x(8), **k),
    lambda **k: gdn.conv_bwd(x(), x(), WEIGHT, d_state=x(2, 3, 8), **k),
    lambda **k: gdn.recur_bwd(x(), x(), x(), STATES, d_gate=x(), **k),
    lambda **k: gdn.recur_bwd(x(), x(), x(), STATES, d_rate=x(8), **k),
])
def test_buffers_of_gradients_that_there_are_not(anywhere, monkeypatch, call):  # noqa: F811
    """A buffer that the call would leave as it was, although it was asked to write there."""
    monkeypatch.setattr(training, "_call", lambda *a: None)      # what passes would be launched
    with pytest.raises(ValueError, match="go with"):
        call()
