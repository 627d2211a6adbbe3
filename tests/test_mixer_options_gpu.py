"""Every optional argument left out by itself, inputs that repeat one row (stride 0), and a
padded call that allocates its output inside a captured graph."""
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from tests.test_mixer_gpu import (BF16, F32, FILL, check_conv, check_norm, check_scan, conv_inputs, draw, gen,
                                  scan_inputs)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(3, 1, 40, 16, 2), (2, 70, 64, 13, 1), (1, 700, 24, 24, 1)])
def test_scan_without_each_option(size, dtype):
    for left_out in (("D",), ("z",), ("dt_bias",), ("h0",), ("D", "z"), ("D", "z", "dt_bias", "h0")):
        i = dict(scan_inputs(*size, dtype, 110), **{k: None for k in left_out})
        y, h = gdn.scan_fwd(**i)
        check_scan(y, h, i)
        alone, none = gdn.scan_fwd(**i, output_final_state=False)
        assert none is None and torch.equal(alone, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 4, 300])
def test_conv_without_each_option(T, dtype):
    for bias, state in ((True, False), (False, True), (False, False)):
        x, w, bi, st, _ = conv_inputs(3, T, 72, 3, dtype, 111, bias, state)
        y, so = gdn.conv_fwd(x, w, bi, st)
        check_conv(y, so, x, w, bi, st, None, "silu")
        alone, none = gdn.conv_fwd(x, w, bi, st, output_final_state=False)
        assert none is None and torch.equal(alone, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(50, 1, 96, 4), (2, 90, 96, 4), (2, 9, 4100, 1)])
def test_group_norm_without_weight_or_bias(size, dtype):
    B, T, C, G = size
    g = gen(112)
    x, w, bi = draw(g, (B, T, C), dtype), torch.randn(C, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    for weight, bias in ((w, None), (None, bi)):
        out = torch.full_like(x, FILL)
        check_norm(gdn.group_norm(x, G, weight, bias, act="silu", out=out), x, G, weight, bias, "silu", None, None)


@pytest.mark.parametrize("T", [1, 3, 130])
def test_rows_of_stride_zero(T):
    """One sequence for a batch, and one token for a sequence."""
    B, D, N = 3, 64, 16
    i = scan_inputs(1, 1, D, N, 1, BF16, 113)
    for rows in ((1, T), (1, 1)):
        j = scan_inputs(*rows, D, N, 1, BF16, 114)
        wide = {k: j[k].expand(B, T, *j[k].shape[2:]) for k in ("x", "dt", "z", "B", "C")}
        dense = {k: v.contiguous() for k, v in wide.items()}
        rest = dict(A=i["A"], D=i["D"], dt_bias=i["dt_bias"], dt_softplus=True)
        w = torch.randn(D, 4, generator=gen(115)).cuda()
        for call in (lambda t: gdn.scan_fwd(**t, **rest), lambda t: gdn.conv_fwd(t["x"], w),
                     lambda t: (gdn.group_norm(t["x"], 4, act="silu", gate=t["z"]),)):
            assert all(torch.equal(a, b) for a, b in zip(call(wide), call(dense)))


def test_padded_calls_replay_from_a_graph():
    T = 300
    x, w, bi, st, _ = conv_inputs(3, T, 64, 4, BF16, 116)
    i = scan_inputs(3, T, 64, 16, 1, BF16, 117)
    n = torch.tensor([T, 0, 7], dtype=torch.int32, device="cuda")
    calls = [lambda: gdn.conv_fwd(x, w, bi, st, lengths=n)[0], lambda: gdn.scan_fwd(**dict(i, lengths=n))[0],
             lambda: gdn.group_norm(x, 4, lengths=n)]
    for call in calls:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for lengths in ([T, 0, 7], [5, T, 1]):       # fewer rows than the replay before wrote
            n.copy_(torch.tensor(lengths, dtype=torch.int32))
            got.fill_(float("nan"))
            graph.replay()
            want = call()
            torch.cuda.synchronize()
            assert torch.equal(got, want) and all((got[b, m:] == 0).all() for b, m in enumerate(lengths))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 40, 900])
def test_nan_and_infinity_stay_in_their_channel(T, dtype, value):
    """One bad value changes its sequence's channel (the norm: its group) from its token on, and
    not a bit of anything else."""
    B, D, G = 6, 72, 9
    t, c = T // 2, 37
    w = torch.randn(D, 3, generator=gen(118)).cuda()
    x, gate = draw(gen(119), (B, T, D), dtype), draw(gen(120), (B, T, D), dtype)
    i = scan_inputs(B, T, D, 16, 1, dtype, 121)
    bad = x.clone()
    bad[2, t, c] = value

    def elsewhere(a, b, *hit):
        same = torch.ones_like(a, dtype=torch.bool)
        same[hit] = False
        return torch.equal(a[same], b[same])

    (y0, s0), (y1, s1) = gdn.conv_fwd(x, w), gdn.conv_fwd(bad, w)
    assert elsewhere(y0, y1, 2, slice(t, t + 3), c) and elsewhere(s0, s1, 2, slice(None), c)
    assert not torch.isfinite(y1[2, t, c])
    (y0, h0), (y1, h1) = gdn.scan_fwd(**dict(i, x=x)), gdn.scan_fwd(**dict(i, x=bad))
    assert elsewhere(y0, y1, 2, slice(t, None), c) and elsewhere(h0, h1, 2, c)
    assert not torch.isfinite(y1[2, t, c])
    g = slice(c // (D // G) * (D // G), (c // (D // G) + 1) * (D // G))
    y0, y1 = gdn.group_norm(x, G, gate=gate, act="silu"), gdn.group_norm(bad, G, gate=gate, act="silu")
    assert elsewhere(y0, y1, 2, slice(None), g) and torch.isnan(y1[2, :, g]).all()
    wide = draw(gen(122), (B, 3, 8192), dtype)
    y0 = gdn.group_norm(wide, 2)
    wide[2, 1, 4100] = value
    y1 = gdn.group_norm(wide, 2)
    assert elsewhere(y0, y1, 2, slice(None), slice(4096, None)) and torch.isnan(y1[2, :, 4096:]).all()
