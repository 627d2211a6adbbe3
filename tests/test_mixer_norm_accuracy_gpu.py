"""The group norm's statistics where rounding shows: means far from zero, and outliers.

u = 2^-24. The mean of a sequence's group is held as a sample of it plus a sum of
differences: the sample's own channel mean, the group's and the cluster's take one rounding
of the mean's size each (3u |mean|), everything else is summed at the size of the
deviations, at most 256 + 64 terms in a row of sizes up to 8 deviations in these inputs
(2560u of a deviation). The variance adds per-piece sums, at most 64 of a set and 256 of a
group in a row, with at most four times the variance in a small set, and three times in a
large one, lost to the point they are taken about: within (3 (67 + 8) + 256 + 16)u, the
deviation within half of that, below 256u."""
import numpy as np
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from oracle import mixer as ref
from tests import mixer_bounds as mb
from tests.test_mixer_gpu import f64, gen

pytestmark = pytest.mark.gpu


def check(x, G, n=None):
    want, v, xhat, size = ref.group_norm(f64(x), G, None, None, 1e-5, "none", None, n)
    bound = 3 * mb.U * size + 2560 * mb.U + abs(xhat) * 260 * mb.U + 2 * mb.U * abs(v)
    lengths = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    mb.check(gdn.group_norm(x, G, lengths=lengths), want, bound, x.dtype)


@pytest.mark.parametrize("size", [(48, 600, 1, 1), (24, 700, 16, 4), (2, 20000, 8, 2), (1, 2300, 1024, 1),
                                  (1, 4500, 255, 1), (12, 40, 4096, 1), (24, 30, 1003, 1), (12, 1, 4100, 2),
                                  (8, 300, 330, 11), (400, 1, 128, 1)])
def test_mean_far_from_zero(size):
    """Deviations of 1 about means of 10^4 to 10^6, so that the mean's roundings lead."""
    B, T, C, G = size
    g = gen(710)
    mean = 10 ** (4 + 2 * torch.rand(B, 1, G, 1, generator=g)) * torch.randn(B, 1, G, 1, generator=g).sign()
    x = (mean + torch.randn(B, T, G, C // G, generator=g)).view(B, T, C).cuda()
    check(x, G)
    if T > 1:
        check(x, G, [max(1, T - 7 * b) for b in range(B)])


@pytest.mark.parametrize("size", [(1, 128, 4096), (1, 128, 1023), (2, 37, 2052), (1, 64, 1024), (3, 1, 4096)])
@pytest.mark.parametrize("value", [180.5, -3.0e4])
def test_outliers_first(size, value):
    """The first value of each thread's share is all there is: what sums are taken about must
    not be that value alone."""
    B, T, C = size
    x = torch.zeros(B, T, C, device="cuda")
    V = 4 if C % 4 == 0 else 1
    x[:, ::16, :256 * V:V] = value
    want, v, xhat, size = ref.group_norm(f64(x), 1, None, None, 1e-5, "none")
    bound = abs(xhat) * 260 * mb.U + 256 * mb.U * size + 2 * mb.U * abs(v)
    mb.check(gdn.group_norm(x, 1), want, bound, x.dtype)


def test_constant_rows_of_wide_groups():
    """No deviation at all: zeros, whatever the value."""
    for value in (0.1, 1e5, -7.3e-6):
        for T, C in ((40, 4096), (3, 1003), (1, 4100), (300, 64), (2300, 1024)):
            x = torch.full((2, T, C), value, device="cuda")
            y = gdn.group_norm(x, 1)
            mean_off = 3 * mb.U * abs(value) / np.sqrt(1e-5)
            assert y.abs().max() <= mean_off
