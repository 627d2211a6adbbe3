"""The sequence-mixer operators measured against their plain forms.

Three operators that surround the gated delta rule in a mixing layer, each for
prompts and (the first two) for single tokens:

* ``conv``: a causal depthwise convolution of a few taps with its activation,
  y[b,t,c] = act(bias[c] + sum_k w[c,k] x[b,t-W+1+k,c]), the tokens before the
  first one taken from a window state;
* ``scan``: the selective state space scan, with Delta = softplus(dt + dt_bias),
  h_t[d,n] = exp(Delta_t[d] A[d,n]) h_{t-1}[d,n] + Delta_t[d] B_t[n] x_t[d] and
  y_t[d] = (sum_n C_t[n] h_t[d,n] + D[d] x_t[d]) silu(z_t[d]);
* ``norm``: group normalisation of channels-last rows with an activation or a gate,
  statistics over a sequence's tokens and a group's channels.

Sizes come from the repository's workloads (16, 32 or 64 heads of 128 channels;
batches of 1, 4, 8 and 256; 1 to 32768 tokens) and from odd ones between them.
``lengths`` (where a case is ragged) holds the valid tokens of each sequence; the
rows at or past it are left as they were, here zeros.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# --------------------------------------------------------------------- cases
def _conv(name, B, T, C, W, dtype, act="silu", bias=True, state=True, ragged=False, strided=False):
    return {"name": name, "op": "conv", "B": B, "T": T, "C": C, "W": W, "dtype": dtype, "act": act,
            "bias": bias, "state": state, "ragged": ragged, "strided": strided}


def _scan(name, B, T, D, N, G, dtype, step=False, gate=True, state=True, ragged=False, strided=True):
    return {"name": name, "op": "scan", "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype,
            "step": step, "gate": gate, "state": state, "ragged": ragged, "strided": strided}


def _norm(name, B, T, C, G, dtype, act="silu", gate=False, ragged=False):
    return {"name": name, "op": "norm", "B": B, "T": T, "C": C, "G": G, "dtype": dtype, "act": act,
            "gate": gate, "ragged": ragged}


def listed():
    return [
        # the convolution of a whole layer's values over the wide batch: 64 heads of 128
        _conv("conv_b8_t8192_c8192", 8, 8192, 8192, 4, "bf16", bias=False, state=False),
        # one half of a fused input projection (rows strided), padded prompts of unequal
        # lengths that continue from earlier windows
        _conv("conv_ragged_b4_t2048_c4096", 4, 2048, 4096, 4, "bf16", ragged=True, strided=True),
        # odd channel count, three taps, 32 bits, no activation
        _conv("conv_f32_b5_t1021_c1003", 5, 1021, 1003, 3, "f32", act="none", ragged=True),
        # one token of 256 sequences: q, k and v of 16 heads of 128 side by side
        _conv("conv_step_b256_c6144", 256, 1, 6144, 4, "bf16"),
        # a batch of prompts through a layer of 4096 channels
        _scan("scan_b4_t2048_d4096", 4, 2048, 4096, 16, 1, "bf16", state=False),
        # one long prompt that continues from a state: few rows, a long serial axis
        _scan("scan_b1_t32768_d2048", 1, 32768, 2048, 16, 1, "bf16"),
        # padded prompts of unequal lengths, an odd state size, two groups, 32 bits
        _scan("scan_f32_b5_t777_d1000_n24", 5, 777, 1000, 24, 2, "f32", ragged=True),
        # one token of 256 sequences
        _scan("scan_step_b256_d4096", 256, 1, 4096, 16, 1, "bf16", step=True),
        # one token of one sequence: latency
        _scan("scan_step_b1_d2048", 1, 1, 2048, 16, 1, "bf16", step=True),
        # the output stage of 32 heads of 128: every token on its own, gated
        _norm("norm_token_n65536_c4096", 65536, 1, 4096, 32, "bf16", gate=True),
        # statistics over whole sequences, 40 channels to a group
        _norm("norm_seq_b4_t4096_c1280", 4, 4096, 1280, 32, "bf16"),
        # odd sizes, padded sequences (one of them empty), 32 bits, no activation
        _norm("norm_f32_b3_t1001_c330", 3, 1001, 330, 11, "f32", act="none", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; every second one a multiple of 8."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(8, n // 8 * 8)


def draw(rng):
    kind = rng.choice(["conv", "conv_step", "scan", "scan_step", "norm_token", "norm_seq"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5
    if kind == "conv":
        B, C, W = _log(rng, 1, 16), _size(rng, 8, 8192), rng.choice([2, 3, 4])
        T = _log(rng, 1, max(1, min(32768, 2 ** 27 // (B * C))))
        c = _conv("", B, T, C, W, dtype, rng.choice(["silu", "none"]), flip(), flip(), flip(), flip())
    elif kind == "conv_step":
        c = _conv("", _log(rng, 1, 512), rng.randint(1, 4), _size(rng, 64, 8192), rng.choice([2, 3, 4]),
                  dtype, rng.choice(["silu", "none"]), flip(), True, False, flip())
    elif kind == "scan":
        B, G, N = _log(rng, 1, 8), rng.choice([1, 1, 2, 4]), rng.choice([4, 8, 13, 16, 16, 24, 32, 64])
        D = G * _size(rng, 8, 4096 // G)
        T = _log(rng, 1, max(1, min(32768, 2 ** 30 // (B * D * N), 2 ** 26 // (B * D))))
        c = _scan("", B, T, D, N, G, dtype, False, flip(), flip(), flip(), flip())
    elif kind == "scan_step":
        G, N = rng.choice([1, 1, 2, 4]), rng.choice([4, 8, 13, 16, 16, 24, 32, 64])
        D = G * _size(rng, 16, 8192 // G)
        B = _log(rng, 1, max(1, min(512, 2 ** 25 // (D * N))))
        c = _scan("", B, rng.randint(1, 4), D, N, G, dtype, True, flip(), True, False, flip())
    elif kind == "norm_token":
        G = rng.choice([1, 4, 16, 32])
        C = G * _size(rng, 8, 4096 // G if G > 1 else 2048)
        B = _log(rng, 1, max(1, min(65536, 2 ** 27 // C)))
        c = _norm("", B, 1, C, G, dtype, rng.choice(["silu", "none", "sigmoid"]), flip())
    else:
        G = rng.choice([1, 4, 11, 32])
        C = G * _log(rng, 1, 64)
        B = _log(rng, 1, 16)
        T = _log(rng, 2, max(2, min(16384, 2 ** 25 // (B * C))))
        c = _norm("", B, T, C, G, dtype, rng.choice(["silu", "none"]), flip(), flip())
    del c["name"]
    return c


def _lengths(case):
    """Valid tokens of each sequence (None: all). A ragged batch has a full sequence and,
    from two sequences on, an empty one; the rest lie between."""
    if not case["ragged"]:
        return None
    B, T = case["B"], case["T"]
    r = random.Random(B * 100003 + T)
    n = [r.randint(0, T) for _ in range(B)]
    n[0] = T
    if B > 1:
        n[B // 2] = 0
    return n


# -------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    td = TYPES[case["dtype"]]
    f32 = dict(dtype=torch.float32, device=dev)

    def randn(*shape):
        return torch.randn(shape, generator=gen, **f32)

    def rand(*shape):
        return torch.rand(shape, generator=gen, **f32)

    def acts(*shape):
        return torch.randn(shape, generator=gen, dtype=td, device=dev)

    n = _lengths(case)
    s = {"case": case,
         "lengths": None if n is None else torch.tensor(n, dtype=torch.int32, device=dev)}
    B, T = case["B"], case["T"]
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        # half of a projection's output, or a tensor of its own
        s["x"] = acts(B, T, 2 * C)[..., C:] if case["strided"] else acts(B, T, C)
        s["weight"] = randn(C, W) * W ** -0.5
        s["bias"] = 0.1 * randn(C) if case["bias"] else None
        s["state"] = acts(B, W - 1, C) if case["state"] else None
        s["y"] = torch.zeros(B, T, C, dtype=td, device=dev)
        s["state_out"] = torch.zeros(B, W - 1, C, dtype=td, device=dev)
    elif case["op"] == "scan":
        D, N, G = case["D"], case["N"], case["G"]
        if case["strided"]:     # x beside z, and B, C behind the low-rank dt, as projections leave them
            s["x"] = acts(B, T, D)
            s["z"] = acts(B, T, 2 * D)[..., D:] if case["gate"] else None
            r = (D + 15) // 16
            proj = acts(B, T, r + 2 * G * N)
            s["B"] = proj[..., r:r + G * N].unflatten(-1, (G, N))
            s["C"] = proj[..., r + G * N:].unflatten(-1, (G, N))
        else:
            s["x"] = acts(B, T, D)
            s["z"] = acts(B, T, D) if case["gate"] else None
            s["B"], s["C"] = acts(B, T, G, N), acts(B, T, G, N)
        s["dt"] = (0.5 * randn(B, T, D)).to(td)
        # decay rates near -1 .. -N; steps of 0.001 .. 0.1 through the softplus
        s["A"] = -torch.arange(1, N + 1, **f32).expand(D, N) * torch.exp(0.1 * randn(D, N))
        step = torch.exp(math.log(1e-3) + rand(D) * (math.log(1e-1) - math.log(1e-3)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["D"] = 1.0 + 0.1 * randn(D)
        s["h0"] = 0.5 * randn(B, D, N) if case["state"] else None
        s["y"] = torch.zeros(B, T, D, dtype=td, device=dev)
        s["h"] = torch.zeros(B, D, N, **f32)
        s["ws"] = None
        if own and not case["step"]:
            from gated_delta_rule_35_gb300 import scan_workspace_bytes
            s["ws"] = torch.empty(scan_workspace_bytes(B, T, D, N, G, td), dtype=torch.uint8, device=dev)
    else:
        C = case["C"]
        # channels of unequal scale and offset
        s["x"] = (randn(B, T, C) * (0.5 + rand(C)) + randn(C)).to(td)
        s["gate"] = acts(B, T, C) if case["gate"] else None
        s["weight"], s["bias"] = 1.0 + 0.1 * randn(C), 0.1 * randn(C)
        s["y"] = torch.zeros(B, T, C, dtype=td, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _act(v, act):
    if act == "none":
        return v
    g = 1.0 / (1.0 + torch.exp(-v))
    return v * g if act == "silu" else g


def _valid(s):
    """[B, T] truth values of the tokens inside their sequences, or None."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["case"]["T"], device=s["lengths"].device)
    return t[None, :] < s["lengths"][:, None]


def _plain_conv(s):
    c = s["case"]
    B, T, C, W = c["B"], c["T"], c["C"], c["W"]
    x = s["x"].float()
    before = x.new_zeros(B, W - 1, C) if s["state"] is None else s["state"].float()
    xp = torch.cat([before, x], 1)
    y = xp[:, :T] * s["weight"][:, 0]
    for k in range(1, W):
        y += xp[:, k:k + T] * s["weight"][:, k]
    if s["bias"] is not None:
        y += s["bias"]
    y = _act(y, c["act"])
    ok = _valid(s)
    if ok is None:
        window = xp[:, T:]
    else:
        y = y * ok[..., None]
        at = s["lengths"].long()[:, None] + torch.arange(W - 1, device=x.device)
        window = torch.gather(xp, 1, at[..., None].expand(B, W - 1, C))
    return {"y": y.to(s["x"].dtype), "state": window.to(s["x"].dtype)}


def _plain_scan(s):
    c = s["case"]
    B, T, D, N, G = c["B"], c["T"], c["D"], c["N"], c["G"]
    h = torch.zeros_like(s["h"]) if s["h0"] is None else s["h0"]
    ok = _valid(s)
    y = torch.empty(B, T, D, dtype=s["x"].dtype, device=h.device)
    block = max(1, min(64, 2 ** 27 // (B * D * N)))
    for t0 in range(0, T, block):
        t1 = min(T, t0 + block)
        x = s["x"][:, t0:t1].float()
        dt = s["dt"][:, t0:t1].float() + s["dt_bias"]
        dt = torch.clamp(dt, min=0.0) + torch.log1p(torch.exp(-torch.abs(dt)))
        if ok is not None:       # a step of length zero keeps the state
            dt = dt * ok[:, t0:t1, None]
        bm = s["B"][:, t0:t1].float().repeat_interleave(D // G, 2)
        cm = s["C"][:, t0:t1].float().repeat_interleave(D // G, 2)
        a = torch.exp(dt[..., None] * s["A"])
        hs = (dt * x)[..., None] * bm
        for i in range(t1 - t0):
            hs[:, i] += a[:, i] * h
            h = hs[:, i]
        o = (hs * cm).sum(-1) + s["D"] * x
        if s["z"] is not None:
            o = o * _act(s["z"][:, t0:t1].float(), "silu")
        if ok is not None:
            o = o * ok[:, t0:t1, None]
        y[:, t0:t1] = o
        h = h.clone()
    return {"y": y, "h": h}


def _plain_norm(s):
    c = s["case"]
    B, T, C, G = c["B"], c["T"], c["C"], c["G"]
    x = s["x"].float().view(B, T, G, C // G)
    ok = _valid(s)
    if ok is None:
        mean = x.mean((1, 3), keepdim=True)
        d = x - mean
        var = (d * d).mean((1, 3), keepdim=True)
    else:
        m = ok[:, :, None, None]
        count = (s["lengths"].clamp(min=1) * (C // G)).float()[:, None, None, None]
        mean = (x * m).sum((1, 3), keepdim=True) / count
        d = x - mean
        var = (d * d * m).sum((1, 3), keepdim=True) / count
    v = (d * torch.rsqrt(var + EPS)).view(B, T, C) * s["weight"] + s["bias"]
    v = v * _act(s["gate"].float(), c["act"]) if s["gate"] is not None else _act(v, c["act"])
    if ok is not None:
        v = v * ok[..., None]
    return {"y": v.to(s["x"].dtype)}


# ------------------------------------------------------------------ the pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm}[c["op"]](s)
    import gated_delta_rule_35_gb300 as gdn
    if c["op"] == "conv":
        y, st = gdn.conv_fwd(s["x"], s["weight"], s["bias"], s["state"], lengths=s["lengths"],
                             act=c["act"], out=s["y"], final_state=s["state_out"])
        return {"y": y, "state": st}
    if c["op"] == "scan":
        if c["step"]:
            y, h = gdn.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["h0"], D=s["D"], z=s["z"],
                                 dt_bias=s["dt_bias"], dt_softplus=True, state_out=s["h"], out=s["y"])
        else:
            y, h = gdn.scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"],
                                dt_bias=s["dt_bias"], dt_softplus=True, h0=s["h0"],
                                lengths=s["lengths"], workspace=s["ws"], out=s["y"],
                                final_state=s["h"])
        return {"y": y, "h": h}
    y = gdn.group_norm(s["x"], c["G"], s["weight"], s["bias"], eps=EPS, act=c["act"], gate=s["gate"],
                       lengths=s["lengths"], out=s["y"])
    return {"y": y}


# ------------------------------------------------------------ what it takes
def work(case):
    """Bytes: every input of the valid tokens read once and every output written once.
    Flops: a multiply-add counts 2, an exponential, logarithm, division or root 1."""
    e = 4 if case["dtype"] == "f32" else 2
    n = _lengths(case)
    tokens = case["B"] * case["T"] if n is None else sum(n)
    if case["op"] == "conv":
        C, W, B = case["C"], case["W"], case["B"]
        windows = B * (W - 1) * C * e * (2 if case["state"] else 1)
        return {"bytes": 2 * tokens * C * e + windows + C * (W + (1 if case["bias"] else 0)) * 4,
                "flops": tokens * C * (2 * W + (4 if case["act"] == "silu" else 0))}
    if case["op"] == "scan":
        D, N, G, B = case["D"], case["N"], case["G"], case["B"]
        state = B * D * N * 4 * (2 if case["state"] else 1)
        rows = tokens * ((4 if case["gate"] else 3) * D + 2 * G * N) * e
        # per state: the rate times the step, its exponential, the input product and two multiply-adds
        return {"bytes": rows + state + D * (N + 2) * 4,
                "flops": tokens * D * (7 * N + 7 + (5 if case["gate"] else 0))}
    C = case["C"]
    return {"bytes": tokens * C * e * (3 if case["gate"] else 2) + 2 * C * 4,
            "flops": tokens * C * (8 + (0 if case["act"] == "none" else 4))}


# ------------------------------------------------------------ in 64 bits
def _gate64(v, act):
    return {"none": lambda: v, "silu": lambda: v / (1 + (-v).exp()),
            "sigmoid": lambda: 1 / (1 + (-v).exp())}[act]()


def exact(case, seed):
    s = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
            for k, v in s.items() if k not in ("y", "h", "state_out")}
    B, T = case["B"], case["T"]
    n = _lengths(case) or [T] * B
    if case["op"] == "conv":
        W, C = case["W"], case["C"]
        y = torch.zeros(B, T, C, dtype=torch.float64, device=s["x"].device)
        st = torch.zeros(B, W - 1, C, dtype=torch.float64, device=s["x"].device)
        for b in range(B):
            old = st[b].clone() if s["state"] is None else wide["state"][b]
            seq = torch.cat([old, wide["x"][b, :n[b]]], 0)
            if n[b]:
                v = (seq.unfold(0, W, 1) * wide["weight"]).sum(-1)
                y[b, :n[b]] = _gate64(v if s["bias"] is None else v + wide["bias"], case["act"])
            st[b] = seq[n[b]:]
        return {"y": y, "state": st}
    if case["op"] == "scan":
        D, N, G = case["D"], case["N"], case["G"]
        if T * B * D * N > 2 ** 31:
            return None
        h = torch.zeros(B, D, N, dtype=torch.float64, device=s["x"].device)
        if s["h0"] is not None:
            h = wide["h0"].clone()
        y = torch.zeros(B, T, D, dtype=torch.float64, device=h.device)
        step = torch.nn.functional.softplus(wide["dt"] + wide["dt_bias"], threshold=40.0)
        lens = torch.tensor(n, device=h.device)
        for t in range(T):
            live = lens > t
            dd = step[:, t].view(B, G, D // G, 1)
            new = torch.exp(dd * wide["A"].view(1, G, D // G, N)) * h.view(B, G, D // G, N)
            new = new + dd * wide["x"][:, t].view(B, G, D // G, 1) * wide["B"][:, t].unsqueeze(2)
            o = torch.einsum("bgdn,bgn->bgd", new, wide["C"][:, t]).reshape(B, D)
            o = o + wide["D"] * wide["x"][:, t]
            h = torch.where(live[:, None, None], new.reshape(B, D, N), h)
            y[:, t] = torch.where(live[:, None], o, y[:, t])
        if s["z"] is not None:
            y *= _gate64(wide["z"], "silu")
        return {"y": y, "h": h}
    C, G = case["C"], case["G"]
    y = torch.zeros(B, T, C, dtype=torch.float64, device=s["x"].device)

    def rows(v, k):      # v [k sequences, tokens, C]
        v = v.unflatten(-1, (G, C // G))
        var, mean = torch.var_mean(v, (1, 3), correction=0, keepdim=True)
        v = ((v - mean) / (var + EPS).sqrt()).flatten(-2)
        return v * wide["weight"] + wide["bias"]

    for b0 in range(0, B, 4096 if T == 1 else 1):
        b1 = min(B, b0 + (4096 if T == 1 else 1))
        m = n[b0]
        if m == 0:
            continue
        v = rows(wide["x"][b0:b1, :m], b1 - b0)
        y[b0:b1, :m] = v * _gate64(wide["gate"][b0:b1, :m], case["act"]) if s["gate"] is not None \
            else _gate64(v, case["act"])
    return {"y": y}
