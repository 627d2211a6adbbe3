"""Sizes that take the kernels' instances for large batches, long runs and large states.
The launch rules of the host code are repeated here where a size stands near their borders,
so that a test says when a changed rule leaves it behind."""
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from tests import mixer_bounds as mb
from tests.test_mixer_gpu import (BF16, F32, FILL, check_conv, check_norm, check_scan, conv_inputs, draw, gen,
                                  ragged, scan_inputs, spoil)

pytestmark = pytest.mark.gpu
SMS = 152


def up(a, b):
    return -(-a // b)


# ------------------------------------------------------------------ convolution
def conv_pieces(C, dtype):
    V = 16 // dtype.itemsize
    return C // V if C % V == 0 else C


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W,T,C", [(4, 1, 6144), (3, 4, 6144), (2, 2, 1003), (4, 3, 1003)])
def test_conv_tokens_of_large_batches(W, T, C, dtype):
    """Four sequences to a thread; the last batch holds two."""
    B = 258
    assert B % 4 == 2 and up(conv_pieces(C, dtype), 128) * up(B, 4) >= 2 * SMS
    for state, lengths, strided, act in ((True, False, False, "silu"), (False, True, False, "none"),
                                         (True, True, True, "sigmoid")):
        x, w, bi, st, n = conv_inputs(B, T, C, W, dtype, 40 + T, state, state, strided, lengths)
        if lengths:
            spoil(x, n)
        out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
        y, so = gdn.conv_fwd(x, w, bi, st, lengths=n, act=act, out=out)
        mb.untouched(y, check_conv(y, so, x, w, bi, st, n, act), FILL)
        if state:
            same = st.clone()
            again, s2 = gdn.conv_fwd(x, w, bi, same, lengths=n, act=act, out=torch.full_like(out, FILL),
                                     final_state=same)
            assert s2 is same and torch.equal(same, so) and torch.equal(again, y)


def conv_run(B, T, C, dtype):
    """Tokens to a thread."""
    run, cv = 64, conv_pieces(C, dtype)
    while run > 8 and up(T, run) * cv * B < SMS * 4 * 128:
        run //= 2
    return run


@pytest.mark.parametrize("B,T,C,dtype,run", [
    (3, 1900, 1003, BF16, 64), (2, 2570, 1003, F32, 64), (4, 4900, 1024, F32, 64), (1, 9801, 2048, BF16, 32),
    (1, 1300, 1003, BF16, 16), (1, 5003, 2048, BF16, 16)])
def test_conv_long_runs(B, T, C, dtype, run):
    """Runs that pass the ring of four turns many times, against the fp64 form."""
    assert conv_run(B, T, C, dtype) == run
    W = 2 + T % 3
    x, w, bi, st, n = conv_inputs(B, T, C, W, dtype, 50, lengths=B > 1)
    act = "silu" if T % 2 else "none"
    out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
    if n is not None:
        spoil(x, n)
    y, so = gdn.conv_fwd(x, w, bi, st, lengths=n, act=act, out=out)
    mb.untouched(y, check_conv(y, so, x, w, bi, st, n, act), FILL)


@pytest.mark.parametrize("C,dtype", [(8192, BF16), (4096, F32)])
def test_conv_of_any_run_gives_the_same_bits(C, dtype):
    """A call of 64-token runs equals calls of 8-token runs on the carried window."""
    B, T, cut = 2, 2600, 100
    assert conv_run(B, T, C, dtype) == 64 and conv_run(1, cut, C, dtype) == 8
    x, w, bi, st, _ = conv_inputs(B, T, C, 4, dtype, 60)
    n = torch.tensor([T, T - 77], dtype=torch.int32, device="cuda")
    out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
    state = st.clone()
    gdn.conv_fwd(x, w, bi, state, lengths=n, out=out, final_state=state)
    for b, m in enumerate(n.tolist()):
        s = st[b:b + 1].clone()
        for t in range(0, m, cut):
            end = min(m, t + cut)
            y, _ = gdn.conv_step(x[b:b + 1, t:end], w, s, bi)
            assert torch.equal(y[0], out[b, t:end])
        assert torch.equal(s[0], state[b]) and (out[b, m:] == FILL).all()


# ------------------------------------------------------------------------- scan
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,D", [(5, 520), (8, 520), (13, 260), (16, 260), (24, 130), (32, 130), (50, 130),
                                 (64, 130), (100, 130), (128, 130)])
def test_scan_tokens_of_large_states_and_batches(N, D, dtype):
    """Four sequences to a thread and several such sets to a block; then one to a thread."""
    NP = next(n for n in (8, 16, 32, 64, 128) if N <= n)
    channels, G = 128 // (NP // 4), 2
    for B in (611, 3):
        blocks, sets = G * up(D // G, channels), up(B, 4)
        assert (blocks * sets > SMS * 7) == (B == 611) and (blocks * sets < 2 * SMS) == (B == 3)
        few = ((1, dict()), (3, dict(lengths=True, gate=False)))
        for T, kw in few if B == 3 else ((1, dict()), (2, dict(strided=True, lengths=True))):
            i = scan_inputs(B, T, D, N, G, dtype, 70 + T, **kw)
            if i["lengths"] is not None:
                for name in ("x", "dt", "z", "B", "C"):
                    if i[name] is not None:
                        spoil(i[name], i["lengths"])
            out = torch.full(i["x"].shape, FILL, dtype=dtype, device="cuda")
            y, h = gdn.scan_fwd(**i, out=out)
            mb.untouched(y, check_scan(y, h, i), FILL)
            again, h2 = gdn.scan_fwd(**i, out=torch.full_like(out, FILL), final_state=i["h0"])
            assert h2 is i["h0"] and torch.equal(h2, h) and torch.equal(again, y)


# ------------------------------------------------------------------- group norm
def norm_inputs(B, T, C, dtype, seed, gated, strided=False):
    """x of mean 3 and deviation 2; strided: rows that start off 16 bytes, C + 3 apart."""
    g = gen(seed)
    x = draw(g, (B, T, C), dtype, strided)
    x.mul_(2).add_(3)
    gate = draw(g, (B, T, C), dtype, strided) if gated else None
    sb, st, _ = x.stride()
    assert not strided or (B == 1 or sb == T * (C + 3)) and (T == 1 or st == C + 3)
    return x, gate, torch.randn(C, generator=g).cuda(), torch.randn(C, generator=g).cuda()


def norm_case(B, T, C, G, dtype, seed, act, gated, lengths, strided=False):
    x, gate, w, bi = norm_inputs(B, T, C, dtype, seed, gated, strided)
    n = ragged(B, T, seed) if lengths else None
    if lengths:
        spoil(x, n)
        if gated:
            spoil(gate, n)
    out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
    check_norm(gdn.group_norm(x, G, w, bi, act=act, gate=gate, lengths=n, out=out), x, G, w, bi, act, gate, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,cg,G", [(3001, 128, 32), (3001, 13, 33), (1501, 512, 16), (1301, 1024, 8)])
def test_group_norm_of_many_tokens(B, cg, G, dtype):
    """Several turns of the row loop, two rows to a turn where a thread keeps few pieces."""
    V = 16 // dtype.itemsize if cg % (16 // dtype.itemsize) == 0 else 1
    lanes = 1
    while lanes < 32 and lanes < cg // V:
        lanes *= 2
    flight = SMS * 8 * 256 // (G * lanes)
    assert 2 * flight < B or (up(cg // V, lanes) > 2 and flight < B)
    norm_case(B, 1, G * cg, G, dtype, 80, "silu", True, False)
    norm_case(B, 1, G * cg, G, dtype, 81, "none", False, True)
    norm_case(B, 1, G * cg, G, dtype, 82, "sigmoid", True, True, strided=True)


@pytest.mark.parametrize("T,C,G,dtype", [(2300, 2048, 1, BF16), (2300, 1024, 1, F32), (2300, 255, 1, BF16),
                                         (140000, 32, 1, BF16), (140000, 32, 2, F32)])
def test_group_norm_of_many_tokens_to_a_thread(T, C, G, dtype):
    """More than the 128 tokens of a set, whatever slices and clusters (of 16 at most) the host
    chooses: several sets, and blocks beyond those that wait in shared memory."""
    V = 16 // dtype.itemsize if C // G % (16 // dtype.itemsize) == 0 else 1
    assert T // 16 // (256 // (C // G // V)) > 128
    norm_case(1, T, C, G, dtype, 90, "silu", False, False)
    norm_case(2, T, C, G, dtype, 91, "silu", True, True)
    x, gate, w, bi = norm_inputs(1, T, C, dtype, 92, True)
    want = gdn.group_norm(x, G, w, bi, gate=gate, act="sigmoid")
    assert gdn.group_norm(x, G, w, bi, gate=gate, act="sigmoid", out=x) is x and torch.equal(x, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(300, 1, 96, 3), (5, 1, 64, 4), (3, 33, 40, 4), (2, 257, 330, 11), (4, 64, 1280, 32),
                                  (1, 4100, 16, 16), (1, 5, 8200, 2), (2, 40, 4100, 1), (2, 1, 12000, 2)])
def test_group_norm_of_strided_rows(size, dtype):
    for k, (act, gated, lengths) in enumerate((("none", False, False), ("silu", False, True), ("silu", True, True))):
        norm_case(*size, dtype, 95 + k, act, gated, lengths, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(5, 1, 256, 4), (2, 37, 128, 4), (2, 21, 8192, 1), (3, 1, 8192, 1)])
def test_group_norm_of_aligned_slices(size, dtype):
    """x and gate side by side in a wider tensor, whole pieces throughout."""
    B, T, C, G = size
    wide = torch.randn(B, T, 3 * C, generator=gen(99)).to(dtype).cuda()
    x, gate = wide[..., C:2 * C], wide[..., 2 * C:]
    out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
    check_norm(gdn.group_norm(x, G, gate=gate, act="silu", out=out), x, G, None, None, "silu", gate, None)
