"""Training a recurrent mixing layer, measured against plain forms: the gated linear
recurrence with its backward pass, layer norm with its backward pass, and the backward
pass of the short convolution.

* ``recur``: per channel, with s = sigmoid(decay), a = exp(-rate s) (or a = s without a
  rate), m = 1, 1 - a or sqrt(1 - a^2),
  h_t = a_t h_{t-1} + m_t sigmoid(gate_t) x_t, y_t = h_t, for prompts, with the states that
  a backward pass starts from, and for single tokens;
* ``recur_bwd``: its gradients from those of y and of the last state;
* ``ln``: y = (x - mean) rstd w + b of every token's channels (or without the mean), with
  the statistics kept; ``ln_bwd``: dx and the sums over tokens that are the gradients of
  w and b;
* ``conv_bwd``: gradients of y[b,t,c] = act(bias[c] + sum_k w[c,k] x[b,t-W+1+k,c]), the
  tokens before the first one taken from a window state.

Sizes come from the repository's workloads (16, 32 or 64 heads of 128 channels; batches of
1, 4, 8 and 256; 1 to 32768 tokens) and from odd ones between them. ``lengths`` (where a
case is ragged) holds the valid tokens of each sequence; the rows at or past it are left
as they were, here zeros.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5
EVERY = 16      # tokens from one kept state of the recurrence to the next


# --------------------------------------------------------------------- cases
def _recur(name, B, T, D, dtype, op="recur", rate=True, gate=True, scaling="root", state=True,
           keep=False, ragged=False, strided=False):
    return {"name": name, "op": op, "B": B, "T": T, "D": D, "dtype": dtype, "rate": rate, "gate": gate,
            "scaling": scaling, "state": state, "keep": keep, "ragged": ragged, "strided": strided}


def _ln(name, B, T, C, dtype, op="ln", center=True, affine=True, ragged=False, strided=False):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "dtype": dtype, "center": center,
            "affine": affine, "ragged": ragged, "strided": strided}


def _conv(name, B, T, C, W, dtype, act="silu", bias=True, state=True, ragged=False, strided=False):
    return {"name": name, "op": "conv_bwd", "B": B, "T": T, "C": C, "W": W, "dtype": dtype, "act": act,
            "bias": bias, "state": state, "ragged": ragged, "strided": strided}


def listed():
    return [
        # a training batch through a layer of 4096 channels, both gates in one projection
        _recur("recur_b4_t2048_d4096", 4, 2048, 4096, "bf16", state=False, keep=True, strided=True),
        # one long prompt that continues from a state: few rows, a long serial axis
        _recur("recur_b1_t32768_d2048", 1, 32768, 2048, "bf16"),
        # one token of 256 sequences
        _recur("recur_step_b256_d4096", 256, 1, 4096, "bf16", op="recur_step"),
        # the training batch's gradients
        _recur("recur_bwd_b4_t2048_d4096", 4, 2048, 4096, "bf16", op="recur_bwd", state=False, strided=True),
        # those of one long sequence that started from a state
        _recur("recur_bwd_b1_t32768_d2048", 1, 32768, 2048, "bf16", op="recur_bwd"),
        # padded sequences of unequal lengths, 32 bits, the decay a sigmoid by itself
        _recur("recur_bwd_f32_b5_t777_d1000", 5, 777, 1000, "f32", op="recur_bwd", rate=False,
               scaling="complement", ragged=True),
        # the norm before a wide layer, its statistics kept
        _ln("ln_b8_t8192_c4096", 8, 8192, 4096, "bf16"),
        # one token of one sequence: latency
        _ln("ln_b1_t1_c2048", 1, 1, 2048, "bf16", center=False),
        # the wide layer's gradients, sums over 65536 tokens among them
        _ln("ln_bwd_b8_t8192_c4096", 8, 8192, 4096, "bf16", op="ln_bwd"),
        # odd sizes, padded sequences (one of them empty), 32 bits
        _ln("ln_bwd_f32_b3_t1001_c1003", 3, 1001, 1003, "f32", op="ln_bwd", ragged=True),
        # a whole layer's values over the wide batch: 64 heads of 128
        _conv("conv_bwd_b8_t8192_c8192", 8, 8192, 8192, 4, "bf16", bias=False, state=False),
        # odd channel count, three taps, 32 bits, no activation, padded
        _conv("conv_bwd_f32_b5_t1021_c1003", 5, 1021, 1003, 3, "f32", act="none", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """Spread over the logarithm; every second one a multiple of 8."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.5 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["recur", "recur", "recur_step", "recur_bwd", "recur_bwd", "ln", "ln_bwd", "ln_bwd",
                     "conv_bwd", "conv_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    flip = lambda: rng.random() < 0.5
    if op == "recur_step":
        B, D = _log(rng, 1, 512), _size(rng, 16, 8192)
        c = _recur("", B, rng.randint(1, 4), D, dtype, op, flip(), flip(),
                   rng.choice(["none", "complement", "root"]), True, False, False, flip())
    elif op in ("recur", "recur_bwd"):
        B, D = _log(rng, 1, 16), _size(rng, 8, 8192)
        T = _log(rng, 1, max(1, min(32768, 2 ** 25 // (B * D))))
        c = _recur("", B, T, D, dtype, op, flip(), flip(), rng.choice(["none", "complement", "root"]), flip(),
                   op == "recur" and flip(), flip(), flip())
    elif op in ("ln", "ln_bwd"):
        B, C = _log(rng, 1, 16), _size(rng, 8, 16384)
        T = _log(rng, 1, max(1, min(32768, 2 ** 27 // (B * C))))
        c = _ln("", B, T, C, dtype, op, flip(), flip(), flip(), flip())
    else:
        B, C, W = _log(rng, 1, 16), _size(rng, 8, 8192), rng.choice([2, 3, 4])
        T = _log(rng, 1, max(1, min(32768, 2 ** 27 // (B * C))))
        c = _conv("", B, T, C, W, dtype, rng.choice(["silu", "none", "sigmoid"]), flip(), flip(), flip(), flip())
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
def _states(case):
    return (case["B"], (case["T"] + EVERY - 1) // EVERY, case["D"])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    td = TYPES[case["dtype"]]
    f32 = dict(dtype=torch.float32, device=dev)
    op, B, T = case["op"], case["B"], case["T"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, **f32)

    def rand(*shape):
        return torch.rand(shape, generator=gen, **f32)

    def acts(*shape):
        return torch.randn(shape, generator=gen, dtype=td, device=dev)

    def zeros(*shape):
        return torch.zeros(shape, dtype=td, device=dev)

    n = _lengths(case)
    s = {"case": case,
         "lengths": None if n is None else torch.tensor(n, dtype=torch.int32, device=dev), "ws": None}
    if op.startswith("recur"):
        D = case["D"]
        if case["strided"]:     # the gates side by side, as one projection leaves them
            both = acts(B, T, 2 * D)
            s["x"], s["decay"], s["gate"] = acts(B, T, D), both[..., :D], both[..., D:]
        else:
            s["x"], s["decay"], s["gate"] = acts(B, T, D), acts(B, T, D), acts(B, T, D)
        if not case["gate"]:
            s["gate"] = None
        if case["rate"]:        # factors of 0.9 to 0.999 a token, to the eighth power at most
            s["rate"] = -8.0 * torch.log(0.9 + 0.099 * rand(D))
        else:                   # a = sigmoid(decay), most of it kept
            s["rate"] = None
            s["decay"] = s["decay"].add_(1.5)
        s["h0"] = randn(B, D) if case["state"] else None
        s["h"] = torch.zeros(B, D, **f32)
        s["y"], s["states"] = zeros(B, T, D), None
        if case["keep"] or op == "recur_bwd":
            s["states"] = torch.zeros(_states(case), **f32)
        if op == "recur_bwd":
            s["dy"] = acts(B, T, D)
            s["dh"] = randn(B, D) if case["state"] else None
            s["dx"], s["ddecay"] = zeros(B, T, D), zeros(B, T, D)
            s["dgate"] = zeros(B, T, D) if case["gate"] else None
            s["drate"] = torch.zeros(D, **f32) if case["rate"] else None
            s["dh0"] = torch.zeros(B, D, **f32)
            if own:             # the states that the step's forward pass has kept (the plain form recomputes)
                import gated_delta_rule_35_gb300 as gdn
                s["ws"] = torch.empty(gdn.recur_bwd_workspace_bytes(B, T, D, td), dtype=torch.uint8, device=dev)
                gdn.recur_fwd(s["x"], s["decay"], s["rate"], s["gate"], case["scaling"], h0=s["h0"],
                              lengths=s["lengths"], out=s["y"], states=s["states"], output_states=True)
    elif op.startswith("ln"):
        C = case["C"]
        # channels of unequal scale and offset; half of a wider tensor where strided
        x = (randn(B, T, C) * (0.5 + rand(C)) + randn(C)).to(td)
        s["x"] = torch.cat([x, x], -1)[..., C:] if case["strided"] else x
        s["weight"] = 1.0 + 0.1 * randn(C) if case["affine"] else None
        s["bias"] = 0.1 * randn(C) if case["affine"] and case["center"] else None
        s["y"], s["stats"] = zeros(B, T, C), torch.zeros(B, T, 2, **f32)
        if op == "ln_bwd":
            s["dy"], s["dx"] = acts(B, T, C), zeros(B, T, C)
            s["dw"] = torch.zeros(C, **f32) if case["affine"] else None
            s["db"] = torch.zeros(C, **f32) if s["bias"] is not None else None
            if own:             # the statistics that the forward pass of the step has kept
                import gated_delta_rule_35_gb300 as gdn
                s["ws"] = torch.empty(gdn.layer_norm_bwd_workspace_bytes(B, T, C, td), dtype=torch.uint8,
                                      device=dev)
                gdn.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, center=case["center"],
                               lengths=s["lengths"], out=s["y"], stats=s["stats"], output_stats=True)
            else:
                s["stats"] = _plain_ln(s)["stats"]
    else:
        C, W = case["C"], case["W"]
        s["x"] = acts(B, T, 2 * C)[..., C:] if case["strided"] else acts(B, T, C)
        s["dy"], s["dx"] = acts(B, T, C), zeros(B, T, C)
        s["weight"] = randn(C, W) * W ** -0.5
        s["bias"] = 0.1 * randn(C) if case["bias"] else None
        s["state"] = acts(B, W - 1, C) if case["state"] else None
        s["dlast"] = acts(B, W - 1, C) if case["state"] else None
        s["dw"] = torch.zeros(C, W, **f32)
        s["db"] = torch.zeros(C, **f32) if case["bias"] else None
        s["dstate"] = zeros(B, W - 1, C) if case["state"] else None
        if own:
            import gated_delta_rule_35_gb300 as gdn
            s["ws"] = torch.empty(gdn.conv_bwd_workspace_bytes(B, T, C, W, td), dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------- plain forms
def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _valid(s):
    """[B, T, 1] truth values of the tokens inside their sequences, or None."""
    if s["lengths"] is None:
        return None
    t = torch.arange(s["case"]["T"], device=s["lengths"].device)
    return (t[None, :] < s["lengths"][:, None])[..., None]


def _inside(v, ok):
    """v with zeros outside the sequences, whatever lies there."""
    return v if ok is None else torch.where(ok, v, torch.zeros((), dtype=v.dtype, device=v.device))


def _factors(s):
    """(sig, a, keep, m, q): sigmoid(decay), the decay factor, 1 - a, the input's factor and
    gate; a token outside its sequence keeps the state (a = 1, no input)."""
    c, ok = s["case"], _valid(s)
    sig = _sigmoid(s["decay"].float())
    if s["rate"] is not None:
        g = -s["rate"] * sig
        a, away = torch.exp(g), -torch.expm1(g)
    else:
        a, away = sig, _sigmoid(-s["decay"].float())
    if c["scaling"] == "root":
        m = torch.sqrt(away * (1.0 + a))
    else:
        m = away if c["scaling"] == "complement" else torch.ones_like(a)
    q = torch.ones_like(a) if s["gate"] is None else _sigmoid(s["gate"].float())
    if ok is not None:
        one = torch.ones((), device=a.device)
        a, m, q = torch.where(ok, a, one), _inside(m, ok), _inside(q, ok)
    return sig, a, away, m, q


def _plain_recur(s, whole=False):
    c, ok = s["case"], _valid(s)
    B, T, D = c["B"], c["T"], c["D"]
    _, a, _, m, q = _factors(s)
    hs = m * q * _inside(s["x"].float(), ok)
    h = torch.zeros(B, D, device=hs.device) if s["h0"] is None else s["h0"]
    first = h
    for a_t, h_t in zip(a.unbind(1), hs.unbind(1)):
        h = h_t.addcmul_(a_t, h)
    out = {"y": _inside(hs, ok).to(s["x"].dtype), "h": h.clone(), "states": None}
    if c["keep"] or whole:
        kept = torch.cat([first[:, None], hs], 1)[:, 0:T:EVERY]
        out["states"] = kept.clone() if ok is None else _inside(kept, ok[:, ::EVERY])
    if whole:
        out["before"] = torch.cat([first[:, None], hs], 1)[:, :T]
    return out


def _plain_recur_bwd(s):
    c, ok = s["case"], _valid(s)
    sig, a, away, m, q = _factors(s)
    x, before = _inside(s["x"].float(), ok), _plain_recur(s, True)["before"]
    lam = _inside(s["dy"].to(torch.float32, copy=True), ok)      # grows to the gradient of h in place
    carry = torch.zeros_like(before[:, 0]) if s["dh"] is None else s["dh"]
    for a_t, lam_t in zip(a.unbind(1)[::-1], lam.unbind(1)[::-1]):
        carry = a_t * lam_t.add_(carry)
    td = s["x"].dtype
    out = {"dx": _inside(lam * m * q, ok).to(td), "dgate": None, "drate": None, "dh0": carry}
    if s["gate"] is not None:
        out["dgate"] = _inside(lam * m * x * q * (1.0 - q), ok).to(td)
    if c["scaling"] == "root":       # of m by the logarithm of a, times m
        dm = -a * a / m.clamp(min=1e-30)
    else:
        dm = -a if c["scaling"] == "complement" else torch.zeros_like(a)
    dlog = lam * (a * before + q * x * dm)
    if s["rate"] is not None:
        out["drate"] = -_inside(dlog * sig, ok).double().sum((0, 1)).float()
        slope = -s["rate"] * sig * _sigmoid(-s["decay"].float())
    else:
        slope = away
    out["ddecay"] = _inside(dlog * slope, ok).to(td)
    return out


def _plain_ln(s):
    c, ok = s["case"], _valid(s)
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True) if c["center"] else torch.zeros_like(x[..., :1])
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    v = d * rstd
    if s["weight"] is not None:
        v = v * s["weight"]
    if s["bias"] is not None:
        v = v + s["bias"]
    return {"y": _inside(v, ok).to(s["x"].dtype), "stats": _inside(torch.cat([mean, rstd], -1), ok)}


def _plain_ln_bwd(s):
    c, ok = s["case"], _valid(s)
    dy, xhat = _inside(s["dy"].float(), ok), (s["x"].float() - s["stats"][..., :1]) * s["stats"][..., 1:]
    xhat = _inside(xhat, ok)
    wdy = dy if s["weight"] is None else dy * s["weight"]
    dx = wdy - xhat * (wdy * xhat).mean(-1, keepdim=True)
    if c["center"]:
        dx = dx - wdy.mean(-1, keepdim=True)
    return {"dx": _inside(dx * s["stats"][..., 1:], ok).to(s["x"].dtype),
            "dw": None if s["weight"] is None else _sum_rows(dy * xhat),
            "db": None if s["bias"] is None else _sum_rows(dy)}


def _sum_rows(v):
    """Sum over batch and tokens, in 64 bits."""
    return torch.stack([r.double().sum(0) for r in v]).sum(0).float()


def _plain_conv_bwd(s):
    c, ok = s["case"], _valid(s)
    B, T, C, W = c["B"], c["T"], c["C"], c["W"]
    x = _inside(s["x"].float(), ok)
    before = x.new_zeros(B, W - 1, C) if s["state"] is None else s["state"].float()
    xp = torch.cat([before, x], 1)
    p = _inside(s["dy"].float(), ok)
    if c["act"] != "none":
        v = xp[:, :T] * s["weight"][:, 0]
        for k in range(1, W):
            v += xp[:, k:k + T] * s["weight"][:, k]
        if s["bias"] is not None:
            v += s["bias"]
        g = _sigmoid(v)
        p = p * (g * (1.0 + v * (1.0 - g)) if c["act"] == "silu" else g * (1.0 - g))
    dxp = torch.zeros_like(xp)
    for k in range(W):
        dxp[:, k:k + T] += p * s["weight"][:, k]
    if s["dlast"] is not None:       # the last window is inputs n .. n + W - 2 of xp
        n = torch.full((B,), T, device=x.device) if ok is None else s["lengths"].long()
        at = n[:, None] + torch.arange(W - 1, device=x.device)
        dxp.scatter_add_(1, at[..., None].expand(B, W - 1, C), s["dlast"].float())
    td = s["x"].dtype
    dx = dxp[:, W - 1:] if ok is None else _inside(dxp[:, W - 1:], ok)
    return {"dx": dx.to(td), "dw": torch.stack([_sum_rows(p * xp[:, k:k + T]) for k in range(W)], -1),
            "db": None if s["bias"] is None else _sum_rows(p),
            "dstate": None if s["state"] is None else dxp[:, :W - 1].to(td)}


# ------------------------------------------------------------------ the pass
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op in ("recur", "recur_step"):
            return _plain_recur(s)
        return {"recur_bwd": _plain_recur_bwd, "ln": _plain_ln, "ln_bwd": _plain_ln_bwd,
                "conv_bwd": _plain_conv_bwd}[op](s)
    import gated_delta_rule_35_gb300 as gdn
    if op == "recur":
        y, h, *kept = gdn.recur_fwd(s["x"], s["decay"], s["rate"], s["gate"], c["scaling"], h0=s["h0"],
                                    lengths=s["lengths"], out=s["y"], final_state=s["h"], states=s["states"],
                                    output_states=c["keep"])
        return {"y": y, "h": h, "states": kept[0] if kept else None}
    if op == "recur_step":
        y, h = gdn.recur_step(s["x"], s["decay"], s["h0"], s["rate"], s["gate"], c["scaling"],
                              state_out=s["h"], out=s["y"])
        return {"y": y, "h": h, "states": None}
    if op == "recur_bwd":
        dx, ddecay, dgate, drate, dh0 = gdn.recur_bwd(
            s["dy"], s["x"], s["decay"], s["states"], s["rate"], s["gate"], c["scaling"],
            d_final_state=s["dh"], lengths=s["lengths"], workspace=s["ws"], dx=s["dx"], d_decay=s["ddecay"],
            d_gate=s["dgate"], d_rate=s["drate"], d_state=s["dh0"])
        return {"dx": dx, "dgate": dgate, "drate": drate, "dh0": dh0, "ddecay": ddecay}
    if op == "ln":
        y, stats = gdn.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, center=c["center"],
                                  lengths=s["lengths"], out=s["y"], stats=s["stats"], output_stats=True)
        return {"y": y, "stats": stats}
    if op == "ln_bwd":
        dx, dw, db = gdn.layer_norm_bwd(s["dy"], s["x"], s["stats"], s["weight"], bias=s["bias"] is not None,
                                        center=c["center"], lengths=s["lengths"], workspace=s["ws"],
                                        dx=s["dx"], d_weight=s["dw"], d_bias=s["db"])
        return {"dx": dx, "dw": dw, "db": db}
    dx, dw, db, dstate = gdn.conv_bwd(s["dy"], s["x"], s["weight"], s["bias"], s["state"], act=c["act"],
                                      d_final_state=s["dlast"], lengths=s["lengths"], workspace=s["ws"],
                                      dx=s["dx"], d_weight=s["dw"], d_bias=s["db"], d_state=s["dstate"])
    return {"dx": dx, "dw": dw, "db": db, "dstate": dstate}


# ------------------------------------------------------------ what it takes
def work(case):
    """Bytes: every input of the valid tokens read once and every output written once.
    Flops: a multiply-add counts 2, an exponential, division or root 1."""
    e = 4 if case["dtype"] == "f32" else 2
    n = _lengths(case) or [case["T"]] * case["B"]
    tokens, op, B = sum(n), case["op"], case["B"]
    if op.startswith("recur"):
        D = case["D"]
        kept = sum((k + EVERY - 1) // EVERY for k in n) * D * 4
        ins = 2 + case["gate"]
        flops = 9 + 5 * case["gate"] + (3 if case["scaling"] == "root" else 1)
        rate = D * 4 * case["rate"]
        if op == "recur_bwd":
            return {"bytes": tokens * D * e * (1 + 2 * ins) + kept + B * D * 4 * (1 + case["state"]) + 2 * rate,
                    "flops": tokens * D * (flops + 14 + 5 * case["gate"])}
        return {"bytes": tokens * D * e * (ins + 1) + kept * case["keep"] + B * D * 4 * (1 + case["state"]) + rate,
                "flops": tokens * D * flops}
    C = case["C"]
    if op.startswith("ln"):
        par = C * 4 * case["affine"] * (1 + case["center"])
        if op == "ln_bwd":
            return {"bytes": tokens * (C * e * 3 + 8) + par + C * 4 * case["affine"], "flops": tokens * C * 15}
        return {"bytes": tokens * (C * e * 2 + 8) + par, "flops": tokens * C * 8}
    W = case["W"]
    windows = 3 * B * (W - 1) * C * e if case["state"] else 0
    act = {"none": 0, "silu": 8, "sigmoid": 6}[case["act"]] + (2 * W if case["act"] != "none" else 0)
    return {"bytes": 3 * tokens * C * e + windows + 2 * C * 4 * (W + case["bias"]),
            "flops": tokens * C * (4 * W + act)}


# ------------------------------------------------------------ in 64 bits
def _scan64(a, u):
    """h_t = a_t h_{t-1} + u_t over axis 1 from h = 0, by doubling, without overwriting
    (autograd goes through it)."""
    step, T = 1, a.shape[1]
    while step < T:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _recur64(c, x, decay, gate, rate, h0):
    """h of one sequence [1, n, D], all in 64 bits."""
    s = torch.sigmoid(decay)
    if rate is None:
        a, away = s, torch.sigmoid(-decay)
    else:
        a, away = torch.exp(-rate * s), -torch.expm1(-rate * s)
    u = x * torch.sigmoid(gate) if gate is not None else x
    if c["scaling"] == "root":
        u = u * (away * (2 - away)).sqrt()
    elif c["scaling"] == "complement":
        u = u * away
    if h0 is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * h0[:, None], u[:, 1:]], 1)
    return _scan64(a, u)


def exact(case, seed):
    s = prepare(case, seed)
    op, B, T = case["op"], case["B"], case["T"]
    n = _lengths(case) or [T] * B
    dev = s["x"].device
    f64 = dict(dtype=torch.float64, device=dev)
    wide = lambda name, *at: None if s.get(name) is None else s[name][at].double()

    def leaf(v):
        return None if v is None else v.clone().requires_grad_()

    def zeros(v):
        return None if v is None else torch.zeros(v.shape, **f64)

    if op in ("recur", "recur_step"):
        out = {"y": zeros(s["y"]), "h": zeros(s["h"]), "states": zeros(s["states"])}
        for b in range(B):
            h0, at = wide("h0", slice(b, b + 1)), (slice(b, b + 1), slice(0, n[b]))
            first = torch.zeros(1, case["D"], **f64) if h0 is None else h0
            if n[b] == 0:
                out["h"][b] = first[0]
                continue
            h = _recur64(case, wide("x", *at), wide("decay", *at), wide("gate", *at), wide("rate"), h0)
            out["y"][b, :n[b]], out["h"][b] = h[0], h[0, -1]
            if out["states"] is not None:
                kept = torch.cat([first, h[0]], 0)[:n[b]:EVERY]
                out["states"][b, :len(kept)] = kept
        return out
    if op == "recur_bwd":
        out = {"dx": zeros(s["dx"]), "dgate": zeros(s["dgate"]), "drate": zeros(s["drate"]),
               "dh0": zeros(s["dh0"]), "ddecay": zeros(s["ddecay"])}
        for b in range(B):
            last, at = wide("dh", b), (slice(b, b + 1), slice(0, n[b]))
            if n[b] == 0:
                if last is not None:
                    out["dh0"][b] = last
                continue
            x, decay, gate, rate = (leaf(wide("x", *at)), leaf(wide("decay", *at)), leaf(wide("gate", *at)),
                                    leaf(wide("rate")))
            h0 = leaf(torch.zeros(1, case["D"], **f64) if s["h0"] is None else wide("h0", slice(b, b + 1)))
            h = _recur64(case, x, decay, gate, rate, h0)
            up = wide("dy", *at).clone()
            if last is not None:
                up[:, -1] += last
            h.backward(up)
            out["dx"][b, :n[b]], out["ddecay"][b, :n[b]], out["dh0"][b] = x.grad[0], decay.grad[0], h0.grad[0]
            if gate is not None:
                out["dgate"][b, :n[b]] = gate.grad[0]
            if rate is not None:
                out["drate"] += rate.grad
        return out
    C = case["C"]
    if op.startswith("ln"):
        w, bias = leaf(wide("weight")), leaf(wide("bias"))
        out = {"y": zeros(s["y"]), "stats": zeros(s["stats"])} if op == "ln" else {"dx": zeros(s["dx"])}
        for b in range(B):
            at = (b, slice(0, n[b]))
            x = leaf(wide("x", *at))
            mean = x.mean(-1, keepdim=True) if case["center"] else x.new_zeros(n[b], 1)
            rstd = ((x - mean).square().sum(-1, keepdim=True) / C + EPS) ** -0.5
            y = (x - mean) * rstd
            y = y if w is None else w * y
            y = y if bias is None else y + bias
            if op == "ln":
                out["y"][at], out["stats"][at] = y.detach(), torch.cat([mean, rstd], -1).detach()
            else:
                y.backward(wide("dy", *at))
                out["dx"][at] = x.grad
        if op == "ln_bwd":
            out["dw"] = None if w is None else w.grad
            out["db"] = None if bias is None else bias.grad
        return out
    W = case["W"]
    w, bias = leaf(wide("weight")), leaf(wide("bias"))
    out = {"dx": zeros(s["dx"]), "dw": None, "db": None, "dstate": zeros(s["dstate"])}
    for b in range(B):
        seq = torch.zeros(W - 1 + n[b], C, **f64)
        if s["state"] is not None:
            seq[:W - 1] = wide("state", b)
        seq[W - 1:] = wide("x", b, slice(0, n[b]))
        seq.requires_grad_()
        v = sum(seq[k:k + n[b]] * w[:, k] for k in range(W))
        v = v if bias is None else v + bias
        if case["act"] != "none":
            v = torch.sigmoid(v) * (v if case["act"] == "silu" else 1.0)
        loss = (v * wide("dy", b, slice(0, n[b]))).sum()
        if s["dlast"] is not None:
            loss = loss + (seq[n[b]:] * wide("dlast", b)).sum()
        loss.backward()
        out["dx"][b, :n[b]] = seq.grad[W - 1:]
        if s["dstate"] is not None:
            out["dstate"][b] = seq.grad[:W - 1]
    out["dw"], out["db"] = w.grad, None if bias is None else bias.grad
    return out
