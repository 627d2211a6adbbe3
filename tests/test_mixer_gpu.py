"""The short convolution, the selective scan and the group norm on the GPU against
their fp64 forms, elementwise within the bounds of mixer_bounds (and, for the scan,
the bound that the fp64 form carries along the recurrence)."""
import ctypes

import numpy as np
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from gated_delta_rule_35_gb300 import mixer, native
from oracle import mixer as ref
from oracle import recurrence
from tests import mixer_bounds as mb
from tests.pins import rel

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FILL = 7.0


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def draw(g, shape, dtype, strided=False):
    """N(0,1) on the GPU; strided: the last part of rows 3 elements wider and an odd one longer."""
    if not strided:
        return torch.randn(shape, generator=g).to(dtype).cuda()
    wide = torch.randn(shape[0], shape[1], int(np.prod(shape[2:])) + 3, generator=g).to(dtype).cuda()
    return wide[..., 3:].unflatten(-1, shape[2:])


def ragged(B, T, seed):
    n = torch.randint(0, T + 1, (B,), generator=gen(seed + 1))
    n[0] = T + 5                # taken as T
    if B > 1:
        n[1] = 0
    if B > 2:
        n[2] = -3               # taken as 0
    return n.to(torch.int32).cuda()


def spoil(t, lengths):
    """NaN in the rows outside the sequences."""
    for b, n in enumerate(ref.clamp_lengths(lengths.tolist(), t.shape[0], t.shape[1])):
        t[b, n:] = float("nan")


# ------------------------------------------------------------------ convolution
def conv_inputs(B, T, C, W, dtype, seed, bias=True, state=True, strided=False, lengths=False):
    g = gen(seed)
    x = draw(g, (B, T, C), dtype, strided)
    w = (torch.randn(C, W, generator=g) * 0.5).cuda()
    bi = (0.1 * torch.randn(C, generator=g)).cuda() if bias else None
    st = draw(g, (B, W - 1, C), dtype) if state else None
    n = ragged(B, T, seed) if lengths else None
    return x, w, bi, st, n


def check_conv(y, so, x, w, bi, st, n, act):
    want, state, v, S = ref.conv(f64(x), f64(w), f64(bi), f64(st), None if n is None else n.tolist(), act)
    mb.check(y, want, mb.conv_bound(want, v, S, w.shape[1], act), x.dtype, "y")
    assert np.array_equal(f64(so), state)
    return want


CONV_SIZES = [(1, 1, 1), (3, 2, 8), (2, 17, 65), (4, 130, 264), (2, 1025, 40), (1, 64, 1003), (3, 3, 2048)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("size", CONV_SIZES)
def test_conv(size, W, dtype):
    B, T, C = size
    act = ["silu", "none", "sigmoid"][(T + W) % 3]
    for strided, lengths, state, bias in ((False, False, False, False), (True, True, True, True),
                                          (False, True, True, False), (True, False, False, True)):
        x, w, bi, st, n = conv_inputs(B, T, C, W, dtype, 100 + W, bias, state, strided, lengths)
        if lengths:
            spoil(x, n)
        out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
        y, so = gdn.conv_fwd(x, w, bi, st, lengths=n, act=act, out=out)
        assert y is out
        mb.untouched(y, check_conv(y, so, x, w, bi, st, n, act), FILL)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv_in_place_steps_equal_the_prompt(dtype):
    x, w, bi, st, _ = conv_inputs(5, 9, 72, 4, dtype, 7)
    whole, last = gdn.conv_fwd(x, w, bi, st)
    state = st.clone()
    for t0, t1 in ((0, 1), (1, 2), (2, 4), (4, 9)):
        y, so = gdn.conv_step(x[:, t0:t1], w, state, bi)
        assert so is state and torch.equal(y, whole[:, t0:t1])
    assert torch.equal(state, last)
    # a long prompt, cut over many blocks, with its state in place
    x, w, bi, st, _ = conv_inputs(2, 3001, 136, 4, dtype, 8)
    whole, last = gdn.conv_fwd(x, w, bi, st)
    state = st.clone()
    y, _ = gdn.conv_fwd(x, w, bi, state, final_state=state)
    assert torch.equal(y, whole) and torch.equal(state, last)


# ------------------------------------------------------------------------- scan
def scan_inputs(B, T, D, N, G, dtype, seed, gate=True, state=True, strided=False, lengths=False,
                soft=True):
    g = gen(seed)
    x, dt = draw(g, (B, T, D), dtype, strided), draw(g, (B, T, D), dtype, strided)
    if not soft:
        dt = dt.abs() * 0.1
    z = draw(g, (B, T, D), dtype, strided) if gate else None
    bm, cm = draw(g, (B, T, G, N), dtype, strided), draw(g, (B, T, G, N), dtype, strided)
    A = (-torch.arange(1, N + 1).float() * torch.exp(0.2 * torch.randn(D, N, generator=g))).cuda()
    skip = torch.randn(D, generator=g).cuda()
    bias = (torch.rand(D, generator=g) * 6 - 7).cuda() if soft else None
    h0 = torch.randn(B, D, N, generator=g).cuda() if state else None
    n = ragged(B, T, seed) if lengths else None
    return dict(x=x, dt=dt, A=A, B=bm, C=cm, D=skip, z=z, dt_bias=bias, dt_softplus=soft, h0=h0, lengths=n)


def scan_ref(i):
    n = i["lengths"]
    return ref.scan(f64(i["x"]), f64(i["dt"]), f64(i["A"]), f64(i["B"]), f64(i["C"]), f64(i["D"]),
                    f64(i["z"]), f64(i["dt_bias"]), i["dt_softplus"], f64(i["h0"]),
                    None if n is None else n.tolist())


def check_scan(y, h, i):
    want, hw, Ey, Eh = scan_ref(i)
    mb.check(h, hw, Eh, F32, "h")
    mb.check(y, want, Ey, i["x"].dtype, "y")
    return want


SCAN_SIZES = [(1, 1, 1, 1, 1), (2, 3, 8, 16, 1), (3, 17, 66, 13, 2), (2, 65, 64, 24, 1), (2, 130, 40, 64, 4),
              (1, 200, 33, 100, 3), (4, 64, 128, 16, 2), (2, 127, 96, 8, 1), (1, 70, 16, 128, 1),
              (2, 40, 130, 4, 1), (1, 31, 264, 16, 1), (2, 33, 48, 1, 1), (1, 20, 70, 2, 2),
              (2, 75, 64, 24, 2), (1, 100, 72, 48, 1), (1, 70, 64, 96, 1), (2, 66, 64, 17, 1), (1, 90, 40, 40, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", SCAN_SIZES)
def test_scan(size, dtype):
    for k, kw in enumerate((dict(gate=False, state=False), dict(strided=True, lengths=True),
                            dict(lengths=True, gate=False), dict(soft=False, state=False))):
        i = scan_inputs(*size, dtype, 200 + k, **kw)
        if i["lengths"] is not None:
            for name in ("x", "dt", "z", "B", "C"):
                if i[name] is not None:
                    spoil(i[name], i["lengths"])
        out = torch.full(i["x"].shape, FILL, dtype=dtype, device="cuda")
        y, h = gdn.scan_fwd(**i, out=out)
        mb.untouched(y, check_scan(y, h, i), FILL)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [(1, 4001, 16, 16, 1), (2, 1500, 24, 24, 2), (1, 2050, 8, 64, 1),
                                  (3, 700, 40, 5, 1), (1, 300, 72, 128, 1)])
def test_scan_long_sequences_of_few_channels(size, dtype):
    """Where the tokens are cut into segments, with the state in place."""
    for kw in (dict(), dict(lengths=True, strided=True)):
        i = scan_inputs(*size, dtype, 300, **kw)
        want = i["h0"].clone()
        y, h = gdn.scan_fwd(**i)
        if kw:
            n = ref.clamp_lengths(i["lengths"].tolist(), size[0], size[1])
            y = y.clone()
            for b in range(size[0]):
                y[b, n[b]:] = 0
        check_scan(y, h, i)
        assert torch.equal(i["h0"], want)
        again, h2 = gdn.scan_fwd(**i, final_state=i["h0"])
        assert h2 is i["h0"] and torch.equal(h2, h)
        for b in range(size[0]):
            nb = ref.clamp_lengths(None if i["lengths"] is None else i["lengths"].tolist(), *size[:2])[b]
            assert torch.equal(again[b, :nb], y[b, :nb])


@pytest.mark.parametrize("T", [1, 7, 120, 1024])
def test_scan_without_a_step_keeps_its_state(T):
    """Delta = 0: exp(0) is 1 exactly, whatever x holds."""
    i = scan_inputs(2, T, 40, 13, 1, F32, 360, soft=False)
    i["dt"].zero_()
    assert torch.equal(gdn.scan_fwd(**i)[1], i["h0"])


def test_scan_grows_across_segments():
    """Delta A > 0 over a whole segment: its factor alone, e^128, is beyond fp32's range, the
    states that it multiplies (0 and 1e-30) stay within."""
    i = scan_inputs(1, 1024, 16, 4, 1, F32, 350, gate=False, soft=False)
    assert gdn.scan_workspace_bytes(1, 1024, 16, 4, 1, F32) >= 16 * 16 * 4 * 4    # 16 segments
    i["dt"].zero_()
    i["dt"][:, 128:192] = 2
    i["x"][:, :900] = 0
    i["dt"][:, 900:] = 0.01
    i["A"] = torch.tensor([1.0, 0.75, 0.5, -1.0]).repeat(16, 1).cuda()
    i["h0"] = 1e-30 * (torch.arange(16) % 2).float()[None, :, None].repeat(1, 1, 4).cuda()
    check_scan(*gdn.scan_fwd(**i), i)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scan_steps_continue_a_prompt(dtype):
    i = scan_inputs(3, 12, 40, 16, 2, dtype, 400)
    want, hw, Ey, Eh = scan_ref(i)
    cut = lambda a, b: {k: v[:, a:b] if k in ("x", "dt", "z", "B", "C") and v is not None else v
                        for k, v in i.items() if k not in ("h0", "lengths")}
    y0, state = gdn.scan_fwd(**cut(0, 7), h0=i["h0"])
    ys = [y0]
    for a, b in ((7, 8), (8, 9), (9, 12)):
        y, s = gdn.scan_step(**cut(a, b), state=state)
        assert s is state
        ys.append(y)
    mb.check(torch.cat(ys, 1), want, Ey, dtype, "y")
    mb.check(state, hw, Eh, F32, "h")


def test_scan_steps_of_extreme_sizes():
    """Delta of 0, tiny, and large (the state forgotten at once); a silent and an
    overflowing gate."""
    D, N = 8, 16
    dt = torch.tensor([-200.0, -60.0, -20.0, -5.0, 0.0, 20.0, 60.0, 200.0]).expand(2, 6, D).contiguous().cuda()
    z = torch.tensor([-200.0, -89.0, -30.0, 0.0, 1.0, 30.0, 89.0, 200.0]).flip(0).expand(2, 6, D).contiguous().cuda()
    i = scan_inputs(2, 6, D, N, 1, F32, 500)
    i.update(dt=dt, z=z, dt_bias=None)
    y, h = gdn.scan_fwd(**i)
    check_scan(y, h, i)


# ------------------------------------------------------------------- group norm
NORM_SIZES = [(1, 1, 1, 1), (5, 1, 64, 4), (300, 1, 96, 3), (7, 1, 1003, 17), (3, 1, 4096, 1), (2, 1, 12000, 2),
              (2, 2, 8, 8), (3, 33, 40, 4), (2, 257, 330, 11), (1, 1500, 640, 32), (4, 64, 1280, 32),
              (2, 300, 72, 1), (1, 5, 8200, 2), (1, 4100, 16, 16), (1, 9000, 24, 2), (1, 300, 3001, 1)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", NORM_SIZES)
def test_group_norm(size, dtype):
    B, T, C, G = size
    for k, (act, gated, affine, strided, lengths) in enumerate((
            ("none", False, False, False, False), ("silu", False, True, True, True),
            ("sigmoid", True, True, False, True), ("silu", True, True, True, False))):
        g = gen(600 + k)
        x = draw(g, (B, T, C), dtype, strided) * 2
        x += 3
        gate = draw(g, (B, T, C), dtype, strided) if gated else None
        w = torch.randn(C, generator=g).cuda() if affine else None
        bi = torch.randn(C, generator=g).cuda() if affine else None
        n = ragged(B, T, 600 + k) if lengths else None
        if lengths:
            spoil(x, n)
            if gated:
                spoil(gate, n)
        out = torch.full((B, T, C), FILL, dtype=dtype, device="cuda")
        y = gdn.group_norm(x, G, w, bi, act=act, gate=gate, lengths=n, out=out)
        check_norm(y, x, G, w, bi, act, gate, n)


def check_norm(y, x, G, w, bi, act, gate, n):
    want, v, xhat, size = ref.group_norm(f64(x), G, f64(w), f64(bi), 1e-5, act, f64(gate),
                                         None if n is None else n.tolist())
    bound = mb.norm_bound(want, v, xhat, size, f64(w), act, f64(gate),
                          None if gate is None else ref.act(f64(gate), act))
    mb.check(y, want, bound, x.dtype, "y")
    mb.untouched(y, want, FILL)


@pytest.mark.parametrize("T", [1, 50])
def test_group_norm_of_far_means_and_in_place(T):
    """The variance is taken about the mean: a mean of 1000 deviations costs only the
    mean's own rounding."""
    g = gen(700)
    x = (1000.0 + torch.randn(4, T, 96, generator=g)).cuda()
    y = torch.full_like(x, FILL)
    check_norm(gdn.group_norm(x, 3, out=y), x, 3, None, None, "none", None, None)
    same = x.clone()
    assert gdn.group_norm(same, 3, out=same) is same and torch.equal(same, y)
    const = torch.full((2, T, 8), 5.0, device="cuda")
    assert (gdn.group_norm(const, 2) == 0).all()


# ------------------------------------------------------- strides of whole pieces
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_slices_of_aligned_projections(dtype):
    """Slices that start and step by whole 16-byte pieces take the wide loads."""
    B, T, D, N = 2, 45, 72, 16
    g = gen(650)
    wide = torch.randn(B, T, 3 * D + 4 * N, generator=g).to(dtype).cuda()
    x, dt, z = wide[..., :D], wide[..., D:2 * D], wide[..., 2 * D:3 * D]
    bm, cm = (wide[..., 3 * D + k * 2 * N:3 * D + (k + 1) * 2 * N].unflatten(-1, (2, N)) for k in (0, 1))
    w = torch.randn(D, 4, generator=g).cuda()
    y, so = gdn.conv_fwd(x, w, act="silu")
    check_conv(y, so, x, w, None, None, None, "silu")
    i = dict(scan_inputs(B, T, D, N, 2, dtype, 651), x=x, dt=dt, z=z, B=bm, C=cm)
    check_scan(*gdn.scan_fwd(**i), i)
    one = dict(i, **{k: i[k][:, 7:8] for k in ("x", "dt", "z", "B", "C")})
    check_scan(*gdn.scan_fwd(**one), one)
    out = torch.full((B, T, D), FILL, dtype=dtype, device="cuda")
    check_norm(gdn.group_norm(x, 3, act="sigmoid", gate=z, out=out), x, 3, None, None, "sigmoid", z, None)


def test_many_sequences_of_one_token():
    """Batches that fill the GPU take several sequences to a thread; the last batch is partial."""
    B, D, N = 1030, 64, 16
    x, w, bi, st, _ = conv_inputs(B, 1, 1000, 4, BF16, 660)
    y, so = gdn.conv_fwd(x, w, bi, st)
    check_conv(y, so, x, w, bi, st, None, "silu")
    n = torch.randint(0, 3, (B,), generator=gen(661)).to(torch.int32).cuda()
    i = dict(scan_inputs(B, 2, 512, N, 2, F32, 662), lengths=n)
    spoil(i["x"], n)
    out = torch.full((B, 2, 512), FILL, device="cuda")
    y, h = gdn.scan_fwd(**i, out=out)
    mb.untouched(y, check_scan(y, h, i), FILL)


# --------------------------------------------------------------- used together
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layer_prompt_then_tokens(dtype):
    """in-projection halves -> convolution -> scan -> group norm over heads with a gate: a
    padded batch of prompts, then tokens, on the carried states; every operator against
    its fp64 form on the inputs it got."""
    B, T, D, N, G = 3, 70, 64, 16, 4
    g = gen(800)
    new = 4
    lengths = torch.tensor([70, 41, 1], dtype=torch.int32).cuda()
    w, bi = (0.5 * torch.randn(D, 4, generator=g)).cuda(), (0.1 * torch.randn(D, generator=g)).cuda()
    i0 = scan_inputs(B, T, D, N, 1, dtype, 801, state=False)
    nw = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    conv_state = torch.zeros(B, 3, D, dtype=dtype, device="cuda")
    h = torch.zeros(B, D, N, device="cuda")
    for call in range(1 + new):
        t = T if call == 0 else 1
        n = lengths if call == 0 else None
        proj = draw(g, (B, t, 2 * D), dtype)
        x, gate = proj[..., :D], proj[..., D:]
        before = conv_state.clone()
        c, _ = gdn.conv_fwd(x, w, bi, conv_state, lengths=n, final_state=conv_state)
        check_conv(c, conv_state, x, w, bi, before, n, "silu")
        i = dict(i0, x=c, lengths=n, z=None, h0=h.clone())
        for name in ("dt", "B", "C"):
            i[name] = i0[name][:, :t] if call == 0 else i0[name][:, call:call + 1]
        y, _ = gdn.scan_fwd(**dict(i, h0=h), final_state=h)
        if n is not None:
            for b in range(B):
                c[b, lengths[b]:] = 0
        check_scan(y, h, i)
        y = y.contiguous()
        if n is not None:
            for b in range(B):
                y[b, lengths[b]:] = 0
        rows = y.view(B * t, 1, D)
        out = gdn.group_norm(rows, G, nw, None, act="silu", gate=gate.reshape(B * t, 1, D))
        check_norm(out, rows, G, nw, None, "silu", gate.reshape(B * t, 1, D), None)


def test_convolution_feeds_the_gated_delta_rule():
    """q, k, v from three slices of one projection through the convolution into
    chunk_fwd, then a token through conv_step and decode_step, against the fp64 forms."""
    B, T, H, K, V = 2, 100, 2, 64, 64
    g = gen(900)
    proj = draw(g, (B, T + 1, H * (2 * K + V)), F32)
    w = (0.5 * torch.randn(proj.shape[-1], 4, generator=g)).cuda()
    gamma = (-torch.rand(B, T + 1, H, generator=g)).cuda()
    beta = torch.rand(B, T + 1, H, generator=g).cuda()
    cuts = [(0, H * K, K), (H * K, 2 * H * K, K), (2 * H * K, proj.shape[-1], V)]
    full, _, _, _ = ref.conv(f64(proj), f64(w))
    want = [full[..., a:b].reshape(B, T + 1, H, n) for a, b, n in cuts]
    norm = [a / np.sqrt((a ** 2).sum(-1, keepdims=True) + 1e-6) for a in want[:2]]
    o_ref, h_ref = recurrence.forward(*norm, want[2], f64(gamma), f64(beta), 1.0, None, chunk=1)
    qkv, states = [], []
    for a, b, n in cuts:
        y, s = gdn.conv_fwd(proj[:, :T, a:b], w[a:b].contiguous())
        qkv.append(y.view(B, T, H, n))
        states.append(s)
    o, h = gdn.chunk_fwd(*qkv, gamma[:, :T].contiguous(), beta[:, :T].contiguous(), raw_g=True,
                         qk_l2norm=True)
    tok = [gdn.conv_step(proj[:, T:, a:b], w[a:b].contiguous(), s)[0].view(B, 1, H, n)
           for (a, b, n), s in zip(cuts, states)]
    o1, h = gdn.decode_step(*tok, gamma[:, T:].contiguous(), beta[:, T:].contiguous(), h, qk_l2norm=True)
    # fp32 chain: the rule's own fp32 tolerance
    assert rel(torch.cat([o, o1], 1).cpu().numpy(), o_ref) < 1e-4 and rel(h.cpu().numpy(), h_ref) < 1e-4


# ------------------------------------------- streams, graphs, far offsets, refusals
def all_calls(dtype=BF16):
    x, w, bi, st, n = conv_inputs(2, 300, 64, 4, dtype, 1, lengths=False)
    i = scan_inputs(1, 2000, 32, 16, 1, dtype, 2)
    g = gen(3)
    u, gate = draw(g, (2, 200, 160), dtype), draw(g, (2, 200, 160), dtype)
    rows = draw(g, (500, 1, 256), dtype)
    return [lambda **k: gdn.conv_fwd(x, w, bi, st, **k), lambda **k: gdn.scan_fwd(**i, **k),
            lambda **k: (gdn.group_norm(u, 8, act="silu", gate=gate, **k),),
            lambda **k: (gdn.group_norm(rows, 2, **k),),
            lambda **k: gdn.conv_fwd(x[:, :1], w, bi, st, **k),
            lambda **k: gdn.scan_fwd(**{a: v[:, :1] if a in ("x", "dt", "z", "B", "C") else v
                                        for a, v in i.items()}, **k)]


def test_calls_repeat_bit_for_bit_on_another_stream_and_from_a_graph():
    side = torch.cuda.Stream()
    for call in all_calls():
        want = call()
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for _ in range(2):
            for t in got:
                t.fill_(0)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_threads_on_streams_of_their_own():
    import threading
    calls = all_calls()
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(5):
            for c, w in zip(calls, want):
                got = c(stream=s)
                s.synchronize()
                bad.extend(1 for a, b in zip(got, w) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad


def test_state_in_place_replays_from_a_graph():
    """A captured token step advances the state at every replay."""
    x, w, bi, st, _ = conv_inputs(4, 3, 64, 4, BF16, 20)
    i = scan_inputs(4, 3, 64, 16, 1, BF16, 21)
    step = {k: i[k][:, :1].clone() if i[k] is not None else None for k in ("x", "dt", "z", "B", "C")}
    rest = dict(A=i["A"], D=i["D"], dt_bias=i["dt_bias"], dt_softplus=True)
    token = x[:, :1].clone()

    def tokens(conv_state, h, run):
        out = []
        for t in range(3):
            token.copy_(x[:, t:t + 1])
            for k in step:
                if step[k] is not None:
                    step[k].copy_(i[k][:, t:t + 1])
            out.append([a.clone() for a in run(conv_state, h)])
        return out

    def run(conv_state, h):
        return gdn.conv_step(token, w, conv_state, bi)[0], gdn.scan_step(**step, **rest, state=h)[0]

    cs, h = st.clone(), i["h0"].clone()
    want = tokens(cs, h, run)
    cs2, h2 = st.clone(), i["h0"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(cs2, h2)
    cs2.copy_(st)
    h2.copy_(i["h0"])

    def replay(*_):
        g.replay()
        return outs

    got = tokens(cs2, h2, replay)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for u, v in zip(got, want) for a, b in zip(u, v))
    assert torch.equal(cs, cs2) and torch.equal(h, h2)


def test_two_graphs_replay_side_by_side():
    """Each captured scan holds its own workspace."""
    i, j = scan_inputs(1, 3000, 16, 16, 1, BF16, 4), scan_inputs(1, 3000, 16, 16, 1, BF16, 5)
    want = [gdn.scan_fwd(**a) for a in (i, j)]
    graphs, got = [], []
    for a in (i, j):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(gdn.scan_fwd(**a))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_beyond_32_bit_offsets():
    """The second sequence starts 2^31 + 64 elements behind the first."""
    far = 2 ** 31 + 64
    for T, C in ((1, 64), (37, 64)):
        buf = torch.empty(far + T * C, dtype=BF16, device="cuda")
        near = draw(gen(10), (2, T, C), BF16)
        x = torch.as_strided(buf, (2, T, C), (far, C, 1))
        x.copy_(near)
        w = torch.randn(C, 4, generator=gen(11)).cuda()
        for a, b in zip(gdn.conv_fwd(x, w), gdn.conv_fwd(near, w)):
            assert torch.equal(a, b)
        assert torch.equal(gdn.group_norm(x, 4, gate=x), gdn.group_norm(near, 4, gate=near))
        i = scan_inputs(2, T, C, 16, 1, BF16, 12)
        bc = x[..., :16].unflatten(-1, (1, 16)), near[..., :16].unflatten(-1, (1, 16))
        far_y = gdn.scan_fwd(**dict(i, x=x, dt=x, z=x, B=bc[0], C=bc[0]))
        for a, b in zip(far_y, gdn.scan_fwd(**dict(i, x=near, dt=near, z=near, B=bc[1], C=bc[1]))):
            assert torch.equal(a, b)
        del buf, x, bc


def test_no_tokens_pass_the_state_through():
    x = torch.empty(2, 0, 16, device="cuda")
    st = torch.randn(2, 3, 16, device="cuda")
    w = torch.randn(16, 4, device="cuda")
    y, so = gdn.conv_fwd(x, w, state=st)
    assert y.shape == (2, 0, 16) and torch.equal(so, st)
    assert (gdn.conv_fwd(x, w)[1] == 0).all()
    h0 = torch.randn(2, 16, 4, device="cuda")
    bc = torch.empty(2, 0, 1, 4, device="cuda")
    A = -torch.rand(16, 4, device="cuda")
    assert torch.equal(gdn.scan_fwd(x, x, A, bc, bc, h0=h0)[1], h0)
    assert (gdn.scan_fwd(x, x, A, bc, bc)[1] == 0).all()
    assert gdn.group_norm(x, 4).shape == (2, 0, 16)


@pytest.mark.parametrize("W,dtype", [(2, BF16), (4, BF16), (3, torch.float32)])
def test_no_tokens_need_no_weight(W, dtype):
    """The C entry's T = 0 copies the window state, with nothing else passed."""
    p = mixer.ConvProblem(3, 0, 24, W, native.DTYPES[dtype], 1, 0, 0)
    st = torch.randn(3, W - 1, 24, device="cuda").to(dtype)
    out = torch.full_like(st, 7)
    s = torch.cuda.current_stream().cuda_stream
    for given, want in ((st, st), (None, torch.zeros_like(st))):
        assert native.lib().gdn_conv_fwd(ctypes.byref(p), None, None, None, given.data_ptr() if given is not None
                                         else None, None, None, out.data_ptr(), s) == native.GDN_OK
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_wrapper_refusals():
    x = torch.zeros(2, 4, 16, device="cuda")
    w = torch.zeros(16, 4, device="cuda")
    st = torch.zeros(2, 3, 16, device="cuda")
    h = torch.zeros(2, 16, 8, device="cuda")
    A = torch.zeros(16, 8, device="cuda")
    bc = torch.zeros(2, 4, 1, 8, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: gdn.conv_fwd(x, w, act="relu")),
        (ValueError, lambda: gdn.conv_fwd(x.transpose(1, 2), w)),
        (ValueError, lambda: gdn.conv_fwd(x, w[:8])),
        (TypeError, lambda: gdn.conv_fwd(x, w.bfloat16())),
        (TypeError, lambda: gdn.conv_fwd(x.half(), w)),
        (ValueError, lambda: gdn.conv_fwd(x, w, state=st[:, :2])),
        (TypeError, lambda: gdn.conv_fwd(x, w, state=st.bfloat16())),
        (TypeError, lambda: gdn.conv_fwd(x, w, lengths=n.long())),
        (ValueError, lambda: gdn.conv_fwd(x, w, lengths=n[:1])),
        (ValueError, lambda: gdn.conv_fwd(x, w, lengths=n.cpu())),
        (ValueError, lambda: gdn.conv_fwd(x, w, out=x[:, :3])),
        (native.GdnError, lambda: gdn.conv_fwd(x, w, out=x)),
        (native.GdnError, lambda: gdn.conv_fwd(x, torch.zeros(16, 5, device="cuda"))),
        (ValueError, lambda: gdn.scan_fwd(x, x, A, bc[:, :3], bc)),
        (TypeError, lambda: gdn.scan_fwd(x, x, A, bc.bfloat16(), bc)),
        (ValueError, lambda: gdn.scan_fwd(x, x, A, bc.transpose(2, 3), bc)),
        (ValueError, lambda: gdn.scan_fwd(x, x, A[:8], bc, bc)),
        (ValueError, lambda: gdn.scan_step(x, x, A, bc, bc, h[:1])),
        (TypeError, lambda: gdn.scan_step(x, x, A, bc, bc, h.bfloat16())),
        (ValueError, lambda: gdn.scan_fwd(x, x[..., :8], A, bc, bc)),
        (native.GdnError, lambda: gdn.scan_fwd(x, x, A, bc, bc, out=x)),
        (native.GdnError, lambda: gdn.group_norm(x, 3)),
        (ValueError, lambda: gdn.group_norm(x, 4, gate=x[:, :2])),
        (ValueError, lambda: gdn.group_norm(x[0], 4)),
        (native.GdnError, lambda: gdn.group_norm(x, 4, gate=x, out=x)),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()
