"""Rows behind a sequence in the outputs that a padded call allocates itself: zeros, so that
an operator without lengths can take them. The rule is one: with g = beta = 0 such a row
leaves its state alone, unless k or v are NaN there."""
import numpy as np
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from oracle import mixer as ref
from oracle import recurrence
from tests.pins import rel
from tests.test_mixer_gpu import conv_inputs, draw, f64, gen, scan_inputs

pytestmark = pytest.mark.gpu


def leave_nan(*like):
    """Freed memory of these tensors' sizes that holds NaN."""
    for t in like:
        torch.full_like(t, float("nan"))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [3, 90])
def test_rows_behind_a_sequence_are_zeros(T, dtype):
    x, w, bi, st, _ = conv_inputs(3, T, 64, 4, dtype, 31)
    i = scan_inputs(3, T, 64, 16, 1, dtype, 32)
    n = torch.tensor([T, 0, 2], dtype=torch.int32, device="cuda")
    calls = [lambda **k: gdn.conv_fwd(x, w, bi, st, **k)[0],
             lambda **k: gdn.scan_fwd(**dict(i, **k))[0],
             lambda **k: gdn.group_norm(x, 4, **k)]
    side = torch.cuda.Stream()
    for call in calls:
        given = call(lengths=n, out=torch.full_like(x, 7))
        for k in ({}, {"stream": side}):
            torch.cuda.synchronize()
            leave_nan(x)
            y = call(lengths=n, **k)
            torch.cuda.synchronize()
            for b, m in enumerate(n.tolist()):
                assert torch.equal(y[b, :m], given[b, :m])
                assert (y[b, m:] == 0).all() and (given[b, m:] == 7).all()


def test_padded_convolution_feeds_the_gated_delta_rule():
    B, T, H, K, V = 3, 100, 2, 64, 64
    g = gen(910)
    lengths = [100, 37, 0]
    proj = draw(g, (B, T, H * (2 * K + V)), torch.float32)
    w = (0.5 * torch.randn(proj.shape[-1], 4, generator=g)).cuda()
    gamma = (-torch.rand(B, T, H, generator=g)).cuda()
    beta = torch.rand(B, T, H, generator=g).cuda()
    h0 = torch.randn(B, H, K, V, generator=g).cuda()
    for b, m in enumerate(lengths):
        proj[b, m:] = float("nan")
        gamma[b, m:] = beta[b, m:] = 0
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    cuts = [(0, H * K, K), (H * K, 2 * H * K, K), (2 * H * K, proj.shape[-1], V)]
    qkv = []
    for a, b, width in cuts:
        leave_nan(proj[..., a:b].contiguous())
        y, _ = gdn.conv_fwd(proj[..., a:b], w[a:b].contiguous(), lengths=n)
        qkv.append(y.view(B, T, H, width))
    o, h = gdn.chunk_fwd(*qkv, gamma, beta, h0=h0, raw_g=True, qk_l2norm=True)
    full, _, _, _ = ref.conv(f64(proj), f64(w), lengths=lengths)
    for b, m in enumerate(lengths):
        if m == 0:
            assert torch.equal(h[b], h0[b])
            continue
        q, k, v = (full[b:b + 1, :m, lo:hi].reshape(1, m, H, width) for lo, hi, width in cuts)
        q, k = (a / np.sqrt((a ** 2).sum(-1, keepdims=True) + 1e-6) for a in (q, k))
        o64, h64 = recurrence.forward(q, k, v, f64(gamma[b:b + 1, :m]), f64(beta[b:b + 1, :m]), 1.0,
                                      f64(h0[b:b + 1]), chunk=1)
        # fp32 chain: the rule's own fp32 tolerance
        assert rel(o[b:b + 1, :m].cpu().numpy(), o64) < 1e-4 and rel(h[b:b + 1].cpu().numpy(), h64) < 1e-4
