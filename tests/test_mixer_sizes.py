"""Sizes that a problem's 32-bit fields cannot hold are refused, not wrapped. The plans
are made here from CPU tensors, expanded from single elements, as if these were on a
device; no call follows."""
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import mixer, native

FAR = 2 ** 32


def refused(call):
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.status == native.GDN_ERR_UNSUPPORTED


@pytest.fixture
def anywhere(monkeypatch):
    monkeypatch.setattr(mixer, "_x", lambda x, axes=None: (x.shape, x.dtype, x.get_device()))


def ones(*shape, dtype=torch.float32):
    return torch.ones((1,) * len(shape), dtype=dtype).expand(shape)


@pytest.mark.parametrize("sizes", [(1, FAR + 100, 64, 16), (FAR + 1, 4096, 64, 16), (1, 4096, FAR + 64, 16),
                                   (1, 4096, 64, FAR + 16), (1, 4096, 64, 16, FAR + 1), (1, 2 ** 31, 64, 16),
                                   (1, -FAR + 100, 64, 16)])
def test_scan_workspace(sizes):
    refused(lambda: gdn.scan_workspace_bytes(*sizes))


def test_conv(anywhere):
    w = torch.ones(1, 4)
    plan = lambda *shape: mixer._conv_plan(ones(*shape), w, None, None, None, "silu", None, None)
    assert plan(3, 5, 1)[1:] == ((3, 3, 1), -1)
    refused(lambda: plan(1, FAR + 5, 1))
    refused(lambda: plan(FAR + 3, 5, 1))


def test_scan(anywhere):
    def plan(B, T):
        x, bc = ones(B, T, 1), ones(B, T, 1, 1)
        return mixer._scan_plan(x, x, torch.ones(1, 1), bc, bc, None, None, None, False, None, None, None, None)

    assert plan(3, 5)[2:] == ((3, 1, 1), -1)
    refused(lambda: plan(1, FAR + 5))
    refused(lambda: plan(FAR + 3, 5))


def test_group_norm(anywhere):
    plan = lambda groups, *shape: mixer._norm_plan(ones(*shape), groups, None, None, 1e-5, "none", None, None, None)
    assert plan(1, 3, 5, 1)[1] == -1
    refused(lambda: plan(FAR + 1, 3, 5, 1))
    refused(lambda: plan(1, 1, FAR + 5, 1))
    refused(lambda: plan(1, FAR + 3, 5, 1))


@pytest.mark.gpu
def test_group_norm_groups_on_the_gpu():
    x = torch.randn(2, 3, 16, device="cuda")
    refused(lambda: gdn.group_norm(x, FAR + 4))
    refused(lambda: gdn.conv_fwd(x[:1, :1, :1].expand(1, FAR + 5, 1), torch.ones(1, 4, device="cuda")))
