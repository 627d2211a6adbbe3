"""How the gated linear recurrence, layer norm and the gradients are called: as the training step
of a layer, captured and replayed, on side streams, from two threads, on expanded and on very
large tensors, with NaN next to what is looked at."""
import threading

import numpy as np
import pytest
import torch

import gated_delta_rule_35_gb300 as gdn
from oracle import training as ref
from tests.mixer_bounds import check
from tests.pins import rel
from tests.test_mixer_gpu import draw, f64, gen
from tests.test_training_gpu import checked, norm_inputs, recur_inputs

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------ a layer's training step
class Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, n):
        y, stats = gdn.layer_norm(x, w, b, lengths=n, output_stats=True)
        ctx.save_for_backward(x, w, stats, n)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, stats, n = ctx.saved_tensors
        dx, dw, db = gdn.layer_norm_bwd(dy, x, stats, w, bias=True, lengths=n)
        return dx, dw, db, None


class Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, b, n):
        ctx.save_for_backward(x, w, b, n)
        return gdn.conv_fwd(x, w, b, lengths=n, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        x, w, b, n = ctx.saved_tensors
        return (*gdn.conv_bwd(dy, x, w, b, lengths=n)[:3], None)


class Recur(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, decay, rate, gate, h0, n):
        y, h, states = gdn.recur_fwd(x, decay, rate, gate, h0=h0, lengths=n, output_states=True)
        ctx.save_for_backward(x, decay, rate, gate, states, n)
        return y, h

    @staticmethod
    def backward(ctx, dy, dh):
        x, decay, rate, gate, states, n = ctx.saved_tensors
        dx, dd, dg, dr, d0 = gdn.recur_bwd(dy, x, decay, states, rate, gate, d_final_state=dh.contiguous(), lengths=n)
        return dx, dd, dr, dg, d0, None


def layer(p, n, norm, conv, recur):
    """norm -> one projection of four parts -> convolution -> recurrence -> gated output, and a
    number that weighs the output and the last state."""
    D = p["conv_w"].shape[0]
    a = norm(p["x"], p["norm_w"], p["norm_b"], n) @ p["proj"]
    u = conv(a[..., :D], p["conv_w"], p["conv_b"], n)
    y, h = recur(u, a[..., D:2 * D], p["rate"], a[..., 2 * D:3 * D], p["h0"], n)
    out = (y * torch.sigmoid(a[..., 3 * D:])) @ p["out"]
    return (out * p["weigh"]).sum() + (h * p["weigh_h"]).sum()


def plain(lengths):
    """The operators in fp64 by autograd's own rules; tokens behind a sequence are zeros."""
    def inside(v):
        ok = torch.arange(v.shape[1])[None, :, None] < torch.tensor(lengths)[:, None, None]
        return torch.where(ok, v, torch.zeros((), dtype=v.dtype)), ok

    def norm(x, w, b, n):
        return inside(torch.nn.functional.layer_norm(x, x.shape[-1:], w, b))[0]

    def conv(x, w, b, n):
        xp = torch.nn.functional.pad(x, (0, 0, w.shape[1] - 1, 0))
        v = sum(xp[:, k:k + x.shape[1]] * w[:, k] for k in range(w.shape[1])) + b
        return inside(torch.nn.functional.silu(v))[0]

    def recur(x, decay, rate, gate, h0, n):
        g = -rate * torch.sigmoid(decay)
        a, m = torch.exp(g), torch.sqrt(-torch.expm1(2 * g))
        u, h, ys = m * torch.sigmoid(gate) * x, h0, []
        ok = inside(x)[1]
        for t in range(x.shape[1]):
            h = torch.where(ok[:, t], a[:, t] * h + u[:, t], h)
            ys.append(h)
        return inside(torch.stack(ys, 1))[0], h

    return norm, conv, recur


def parameters(B, T, C, D, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return dict(x=r(B, T, C), norm_w=1 + 0.1 * r(C), norm_b=0.1 * r(C), proj=r(C, 4 * D) * C ** -0.5,
                conv_w=0.5 * r(D, 4), conv_b=0.1 * r(D), rate=0.05 + torch.rand(D, generator=g), h0=r(B, D),
                out=r(D, C) * D ** -0.5, weigh=r(B, T, C), weigh_h=r(B, D))


@pytest.mark.parametrize("C,D,lengths", [(96, 128, None), (65, 33, [150, 0, 77])])
def test_gradients_of_a_layer(C, D, lengths):
    """fp32, against fp64: each of the operators is within some 1e-6 of its values, the products
    of the projections (D and C terms, TF32 off) too, six of them in a row: 1e-4 leaves an order."""
    B, T = 3, 150
    host = parameters(B, T, C, D, 900)
    dev = {k: v.cuda().requires_grad_(k not in ("weigh", "weigh_h")) for k, v in host.items()}
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    loss = layer(dev, n, Norm.apply, Conv.apply, Recur.apply)
    loss.backward()
    wide = {k: v.double().requires_grad_(k not in ("weigh", "weigh_h")) for k, v in host.items()}
    want = layer(wide, None, *plain(lengths or [T] * B))
    want.backward()
    scale = float((wide["weigh"] ** 2).sum().sqrt())
    assert abs(float(loss.detach()) - float(want.detach())) < 1e-4 * scale
    for k, v in wide.items():
        if v.requires_grad:
            assert rel(dev[k].grad.cpu().numpy(), v.grad.numpy()) < 1e-4, k


def test_gradients_of_a_layer_by_differences():
    """Along a random direction of all parameters at once: the loss is a sum of 28800 terms of size
    1, off by 28800^(1/2) 2^-24 or so, 1e-5; a step of 1e-2 leaves 1e-3 of it in the quotient, and its
    third derivative as much again times the square of the step."""
    host = parameters(2, 100, 48, 32, 901)
    dev = {k: v.cuda().requires_grad_(k not in ("weigh", "weigh_h")) for k, v in host.items()}
    run = lambda p: layer(p, None, Norm.apply, Conv.apply, Recur.apply)
    run(dev).backward()
    g = gen(902)
    way = {k: torch.randn(v.shape, generator=g).cuda() * (0.1 if k == "rate" else 1) for k, v in dev.items()
           if v.requires_grad}
    size = sum(float((w ** 2).sum()) for w in way.values()) ** 0.5
    slope = sum(float((dev[k].grad * w).sum()) for k, w in way.items()) / size
    step = 1e-2
    moved = lambda s: float(run({k: v.detach() + s * way[k] / size if k in way else v.detach()
                                 for k, v in dev.items()}))
    grad = sum(float((dev[k].grad ** 2).sum()) for k in way) ** 0.5
    assert abs((moved(step) - moved(-step)) / (2 * step) - slope) < 5e-3 * grad


# ---------------------------------------------------------------------- the calls
def calls(dtype, D=72, T=150, seed=910):
    """(call, inputs) of every operator; a call takes its inputs and outputs of its own."""
    i = recur_inputs(3, T, D, dtype, seed, lengths=True)
    x, w, b, dy, _ = norm_inputs(3, T, D, dtype, seed + 1)
    cw = torch.randn(D, 4, generator=gen(seed + 2)).cuda()
    n = i["lengths"]
    _, _, states = gdn.recur_fwd(**i, output_states=True)
    _, stats = gdn.layer_norm(x, w, b, output_stats=True)
    no_state = {k: v for k, v in i.items() if k != "h0"}
    last = torch.randn(3, 3, D, generator=gen(seed + 3)).to(dtype).cuda()
    return [lambda **k: gdn.recur_fwd(**i, output_states=True, **k),
            lambda **k: gdn.recur_step(i["x"][:, :3], i["decay"][:, :3], i["h0"], i["rate"], i["gate"][:, :3],
                                       state_out=torch.empty_like(i["h0"]), **k),
            lambda **k: gdn.recur_bwd(dy, states=states, **no_state, **k),
            lambda **k: gdn.layer_norm(x, w, b, lengths=n, output_stats=True, **k),
            lambda **k: gdn.layer_norm_bwd(dy, x, stats, w, bias=True, lengths=n, **k),
            lambda **k: gdn.conv_bwd(dy, x, cw, b, last, d_final_state=last, lengths=n, **k)]


def same(a, b):
    """Bit for bit, NaN (behind sequences whose inputs hold it) included."""
    for u, v in zip(a, b):
        assert (u is None) == (v is None)
        if u is not None:
            assert torch.equal(u.nan_to_num(7.0), v.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [72, 65])
def test_streams(D, dtype):
    side = torch.cuda.Stream()
    for call in calls(dtype, D):
        want = call()
        torch.cuda.synchronize()
        got = call(stream=side)
        with torch.cuda.stream(side):
            again = call()
        side.synchronize()
        same(got, want)
        same(again, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    """All operators in one graph, replayed on other inputs in the same buffers."""
    i = recur_inputs(2, 140, 136, dtype, 920)
    x, w, b, dy, _ = norm_inputs(2, 140, 136, dtype, 921)
    cw = torch.randn(136, 3, generator=gen(922)).cuda()
    inputs = [i["x"], i["decay"], i["gate"], x, dy]

    def step():
        y, h, states = gdn.recur_fwd(**i, output_states=True)
        no_state = {k: v for k, v in i.items() if k != "h0"}
        out = [y, h, states, *gdn.recur_bwd(dy, states=states, **no_state)]
        z, stats = gdn.layer_norm(x, w, b, output_stats=True)
        out += [z, stats, *gdn.layer_norm_bwd(dy, x, stats, w, bias=True)]
        return out + [v for v in gdn.conv_bwd(dy, x, cw, b) if v is not None]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (923, 924):
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in captured]
        same(got, step())


def test_two_graphs_with_a_workspace_each():
    x, w, b, dy, _ = norm_inputs(2, 700, 264, BF16, 930)
    other = torch.randn(2, 700, 264, generator=gen(931)).bfloat16().cuda()
    _, stats = gdn.layer_norm(x, w, b, output_stats=True)
    need = gdn.layer_norm_bwd_workspace_bytes(2, 700, 264)
    graphs, outs = [], []
    for d in (dy, other):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        gdn.layer_norm_bwd(d, x, stats, w, bias=True, workspace=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(gdn.layer_norm_bwd(d, x, stats, w, bias=True, workspace=ws))
        graphs.append((g, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for d, out in zip((dy, other), outs):
        same(out, gdn.layer_norm_bwd(d, x, stats, w, bias=True))


def test_two_threads():
    work = [calls(BF16, 72), calls(F32, 65, 40)]
    want = [[c() for c in w] for w in work]
    torch.cuda.synchronize()
    failed = []

    def go(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                with torch.cuda.stream(s):
                    got = [c() for c in work[k]]
                s.synchronize()
                for a, b in zip(got, want[k]):
                    same(a, b)
        except Exception as e:       # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=go, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_two_threads_on_one_kernel():
    """Calls of other sizes on the same kernels, whose blocks take other amounts of shared memory."""
    work = [calls(BF16, 72, T, seed=913) for T in (20, 700)] + [calls(BF16, D, 40, seed=914) for D in (33, 257)]
    want = [[c() for c in w] for w in work]
    torch.cuda.synchronize()
    failed = []

    def go(k):
        try:
            s = torch.cuda.Stream()
            for _ in range(40):
                with torch.cuda.stream(s):
                    got = [c() for c in work[k]]
                s.synchronize()
                for a, b in zip(got, want[k]):
                    same(a, b)
        except Exception as e:       # noqa: BLE001 (reported below)
            failed.append(e)

    threads = [threading.Thread(target=go, args=(k,)) for k in range(len(work))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


def test_workspaces_are_checked():
    x = torch.randn(2, 40, 64, device="cuda")
    w, st, stats = torch.ones(64, 4, device="cuda"), torch.zeros(2, 3, 64, device="cuda"), torch.ones(2, 40, 2, device="cuda")
    for call in (lambda ws: gdn.recur_bwd(x, x, x, st, workspace=ws),
                 lambda ws: gdn.layer_norm_bwd(x, x, stats, w[:, 0].contiguous(), workspace=ws),
                 lambda ws: gdn.conv_bwd(x, x, w, workspace=ws)):
        for ws in (torch.empty(8, dtype=torch.uint8, device="cuda"), torch.empty(1 << 20, device="cuda"),
                   torch.empty(1 << 20, dtype=torch.uint8)):
            with pytest.raises(ValueError):
                call(ws)


# ------------------------------------------------------------------- the tensors
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D", [72, 65, 7])
def test_expanded_inputs(D, dtype):
    """Rows of stride 0, as the gradient of a sum has them, and one row for all tokens."""
    B, T = 2, 45
    row = lambda seed: torch.randn(1, 1, D, generator=gen(seed)).to(dtype).cuda().expand(B, T, D)
    i = recur_inputs(B, T, D, dtype, 940)
    i["decay"] = row(941)
    dy, x = row(942), row(943)
    whole = {k: v.contiguous() if k == "decay" else v for k, v in i.items()}
    _, _, states = gdn.recur_fwd(**i, output_states=True)
    same(gdn.recur_fwd(**i, output_states=True), gdn.recur_fwd(**whole, output_states=True))
    for k in (i, whole):
        k.pop("h0")
    near = lambda a, b: check(a, f64(b), 2.0 ** -20 * float(abs(b.float()).max()), a.dtype)
    for a, b in zip(gdn.recur_bwd(dy, states=states, **i), gdn.recur_bwd(dy.contiguous(), states=states, **whole)):
        near(a, b)
    w = torch.rand(D, generator=gen(944)).cuda()
    y, stats = gdn.layer_norm(x, w, output_stats=True)
    near(y, gdn.layer_norm(x.contiguous(), w))
    for a, b in zip(gdn.layer_norm_bwd(dy, x, stats, w, bias=True),
                    gdn.layer_norm_bwd(dy.contiguous(), x.contiguous(), stats, w, bias=True)):
        near(a, b)
    cw = torch.randn(D, 4, generator=gen(945)).cuda()
    for a, b in zip(gdn.conv_bwd(dy, x, cw, w)[:3], gdn.conv_bwd(dy.contiguous(), x.contiguous(), cw, w)[:3]):
        near(a, b)


@pytest.mark.parametrize("offset", [0, 1, 2, 3, 5, 7])
def test_every_alignment_in_bf16(offset):
    """Slices at every distance from a 16-byte boundary, the first and last rows of their memory."""
    B, T, D = 2, 37, 130
    g = gen(950 + offset)
    cut = lambda: torch.randn(B * T * (D + 5) + offset, generator=g).bfloat16().cuda()[offset:] \
        .as_strided((B, T, D), (T * (D + 5), D + 5, 1), offset)
    x, decay, gate, dy = cut(), cut(), cut(), cut()
    rate = torch.rand(D, generator=g).cuda()
    y, h, states = gdn.recur_fwd(x, decay, rate, gate, output_states=True)
    want, bound, _ = ref.recur(f64(x), f64(decay), f64(rate), f64(gate))
    checked(dict(y=y, h=h, states=states), want, bound, dict(y=BF16))
    got = gdn.recur_bwd(dy, x, decay, states, rate, gate)
    want, bound = ref.recur_bwd(f64(dy), f64(x), f64(decay), f64(rate), f64(gate))
    checked(dict(zip(("dx", "d_decay", "d_gate", "d_rate", "d_state"), got)), want, bound,
            dict(dx=BF16, d_decay=BF16, d_gate=BF16))
    w = torch.rand(D, generator=g).cuda()
    y, stats = gdn.layer_norm(x, w, output_stats=True)
    want, bound = ref.layer_norm(f64(x), f64(w))
    checked(dict(y=y, stats=stats), want, bound, dict(y=BF16))
    want, bound = ref.layer_norm_bwd(f64(dy), f64(x), f64(w))
    checked(dict(zip(("dx", "d_weight", "d_bias"), gdn.layer_norm_bwd(dy, x, stats, w, bias=True))), want, bound,
            dict(dx=BF16))
    cw = torch.randn(D, 4, generator=g).cuda()
    want, bound = ref.conv_bwd(f64(dy), f64(x), f64(cw), f64(w))
    checked(dict(zip(("dx", "d_weight", "d_bias"), gdn.conv_bwd(dy, x, cw, w))), {k: want[k] for k in (
        "dx", "d_weight", "d_bias")}, bound, dict(dx=BF16))


@pytest.mark.parametrize("D", [72, 65])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_stays_where_it_belongs(dtype, D):
    B, T = 3, 150
    i = recur_inputs(B, T, D, dtype, 960)
    dy = draw(gen(961), (B, T, D), dtype)
    w, cw = torch.rand(D, generator=gen(962)).cuda(), torch.randn(D, 4, generator=gen(963)).cuda()
    x = i["x"]
    h0 = i.pop("h0")

    def all_of():
        y, h, states = gdn.recur_fwd(**i, h0=h0, output_states=True)
        z, stats = gdn.layer_norm(x, w, output_stats=True)
        return (y, h, gdn.recur_bwd(dy, states=states, **i), z, gdn.layer_norm_bwd(dy, x, stats, w, bias=True),
                gdn.conv_bwd(dy, x, cw, w))

    clean = all_of()
    b, t, c = 1, 20, 4
    x[b, t, c] = float("nan")
    y, h, (dx, dd, dg, dr, d0), z, (ldx, ldw, ldb), (cdx, cdw, cdb, _) = all_of()
    ok = torch.ones(B, T, D, dtype=torch.bool, device="cuda")

    def but(mask, got, want):
        assert torch.equal(got[mask], want[mask])

    here = ok.clone()
    here[b, t:, c] = False
    but(here, y, clean[0])
    but(here[:, -1], h, clean[1])
    assert torch.isnan(y[b, t:, c]).all()
    all_tokens = ok.clone()
    all_tokens[b, :, c] = False
    for got, want in zip((dx, dd, dg), clean[2]):
        but(all_tokens, got, want)
    but(torch.arange(D, device="cuda") != c, dr, clean[2][3])
    row = ok.clone()
    row[b, t] = False
    but(row, z, clean[3])
    but(row, ldx, clean[4][0])
    assert torch.equal(ldb, clean[4][2]) and torch.isnan(ldw).all() and torch.isnan(z[b, t]).all()
    near = ok.clone()
    near[b, t - 3:t + 4, c] = False         # what the values before the activation that it is in give
    but(near, cdx, clean[5][0])
    other = torch.arange(D, device="cuda") != c
    but(other, cdw, clean[5][1])
    but(other, cdb, clean[5][2])


# What a sequence ends with need not be finite for its gradients to be: its last input, whose factor
# is 1, reaches none of them but its gate's.
@pytest.mark.parametrize("D", [72, 65])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_last_input_that_is_not_finite(value, dtype, D):
    B, T = 3, 150
    i = recur_inputs(B, T, D, dtype, 965, scaling="none")
    i["lengths"] = torch.tensor([150, 20, 97], dtype=torch.int32, device="cuda")
    dy = draw(gen(966), (B, T, D), dtype)

    def gradients():
        _, _, states = gdn.recur_fwd(**i, output_states=True)
        return gdn.recur_bwd(dy, states=states, **{n: v for n, v in i.items() if n != "h0"})

    clean = gradients()
    for b, n in enumerate(i["lengths"].tolist()):
        i["x"][b, n - 1] = value
    dx, d_decay, _, d_rate, d_state = gradients()
    for got, want in zip((dx, d_decay, d_rate, d_state), (clean[0], clean[1], clean[3], clean[4])):
        assert torch.isfinite(want).all() and torch.equal(got, want)


def test_beyond_32_bits():
    """Tensors of more than 2^31 values: the last sequence as if it were alone."""
    B, T, D = 5, 65536, 8192
    assert B * T * D > 2 ** 31
    x = torch.empty(B, T, D, dtype=BF16, device="cuda")
    for b in range(B):
        x[b] = torch.randn(T, D, generator=torch.Generator("cuda").manual_seed(b), device="cuda", dtype=BF16)
    rate = (0.01 + torch.rand(D, generator=gen(970))).cuda()
    close = lambda a, b: check(a, f64(b), 2.0 ** -8 * 0.02 * float(abs(b.float()).max()), a.dtype)
    y, h, states = gdn.recur_fwd(x, x, rate, x, output_states=True)
    last = x[-1:].clone()
    y1, h1, st1 = gdn.recur_fwd(last, last, rate, last, output_states=True)
    close(y[-1:, -40:], y1[:, -40:])
    close(h[-1:], h1)
    del y
    dx, dd, dg, _, d0 = gdn.recur_bwd(x, x, x, states, rate, x)
    dx1, dd1, dg1, _, d01 = gdn.recur_bwd(last, last, last, st1, rate, last)
    for a, b in ((dx, dx1), (dd, dd1), (dg, dg1)):
        close(a[-1:, -40:], b[:, -40:])
        close(a[-1:, :40], b[:, :40])
    close(d0[-1:], d01)
    del dx, dd, dg, states, st1, dx1, dd1, dg1
    w = torch.rand(D, generator=gen(971)).cuda()
    y, stats = gdn.layer_norm(x, w, output_stats=True)
    y1, stats1 = gdn.layer_norm(last, w, output_stats=True)
    assert torch.equal(y[-1:], y1) and torch.equal(stats[-1:], stats1)
    dx = gdn.layer_norm_bwd(x, x, stats, w)[0]
    assert torch.equal(dx[-1:], gdn.layer_norm_bwd(last, last, stats1, w)[0])
    del y, y1
    cw = torch.randn(D, 4, generator=gen(972)).cuda()
    dx = gdn.conv_bwd(x, x, cw, dx=dx)[0]
    assert torch.equal(dx[-1:], gdn.conv_bwd(last, last, cw)[0])
