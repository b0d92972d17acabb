"""The operators around the SSD layer, as they are measured: the short causal
convolution, the selective scan with a decay per (channel, state), and the
norm and position rotation of B and C, each for prompts, training and single
tokens.

``run`` computes them in their plain form (elementary torch operations in
fp32, angles in fp64, one rounding at the end) or, where ``own`` is true,
through the library's entry points.  ``exact`` computes them in fp64 from
their definitions, the recurrences token by token.
"""
import math

import torch

own = False

EPS = 1e-5          # under the square root of the norm


# ------------------------------------------------------------------ cases
def listed():
    return [
        # x, B and C channels (24 * 64 + 2 * 128) of the 130M layer: prompts of
        # different lengths in a padded batch, the conv state kept for decoding
        dict(name="conv_prompt", op="conv", form="fwd", batch=8, seqlen=2048, channels=1792,
             width=4, dtype="bf16", ragged=True),
        # the 2.7B layer's 80 * 64 + 2 * 128 channels, forward and backward: the
        # largest, far beyond L2
        dict(name="conv_train", op="conv", form="train", batch=4, seqlen=8192, channels=5376,
             width=4, dtype="bf16", ragged=False),
        # one token of 256 sequences at the 2.7B layer: latency
        dict(name="conv_token", op="conv", form="step", batch=256, seqlen=1, channels=5376,
             width=4, dtype="bf16", ragged=False),
        # 1536 channels (24 * 64) with 16 states each: prompts of different lengths
        dict(name="scan_prompt", op="scan", form="fwd", batch=8, seqlen=2048, channels=1536,
             dstate=16, groups=1, dtype="bf16", gate=True, ragged=True),
        # one long document: few channels, many tokens
        dict(name="scan_long", op="scan", form="fwd", batch=1, seqlen=32768, channels=1536,
             dstate=16, groups=1, dtype="bf16", gate=True, ragged=False),
        # a training step's scan, 5120 channels (80 * 64): the largest scan
        dict(name="scan_train", op="scan", form="train", batch=4, seqlen=2048, channels=5120,
             dstate=16, groups=1, dtype="bf16", gate=True, ragged=False),
        # fp32, odd sizes, groups, entering states and no gate: a small experiment
        dict(name="scan_train_f32", op="scan", form="train", batch=2, seqlen=777, channels=600,
             dstate=24, groups=3, dtype="f32", gate=False, ragged=False),
        # one token of 256 sequences: the states stream through once
        dict(name="scan_token", op="scan", form="step", batch=256, seqlen=1, channels=5120,
             dstate=16, groups=1, dtype="bf16", gate=True, ragged=False),
        # one token of one sequence: latency alone
        dict(name="scan_token_one", op="scan", form="step", batch=1, seqlen=1, channels=1536,
             dstate=16, groups=1, dtype="bf16", gate=True, ragged=False),
        # B and C of eight groups over the 2.7B layer's tokens, half the pairs turned
        dict(name="rotate_prompt", op="rotate", form="fwd", batch=4, seqlen=8192, groups=8,
             dstate=128, rotary=64, dtype="bf16", interleaved=False, far=False),
        # the same operator's training step at the 130M layer's tokens
        dict(name="rotate_train", op="rotate", form="train", batch=8, seqlen=2048, groups=8,
             dstate=128, rotary=128, dtype="bf16", interleaved=True, far=False),
        # one token of 256 sequences, each far along its document
        dict(name="rotate_token", op="rotate", form="fwd", batch=256, seqlen=1, groups=1,
             dstate=128, rotary=128, dtype="bf16", interleaved=False, far=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("conv", "conv", "scan", "scan", "scan", "rotate"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "conv":
        form = rng.choice(("fwd", "train", "step"))
        c = dict(op=op, form=form, batch=_log_int(rng, 1, 256 if form == "step" else 8),
                 seqlen=1 if form == "step" else _log_int(rng, 2, 8192),
                 channels=_log_int(rng, 32, 5376), width=rng.choice((2, 3, 4, 4, 4)), dtype=dtype,
                 ragged=form == "fwd" and rng.random() < 0.5)
        while c["batch"] * c["seqlen"] * c["channels"] > 6e7:
            c["seqlen"] = max(1, c["seqlen"] // 2)
        return c
    if op == "scan":
        form = rng.choice(("fwd", "train", "step"))
        groups = rng.choice((1, 1, 1, 2, 3))
        c = dict(op=op, form=form, batch=_log_int(rng, 1, 256 if form == "step" else 8),
                 seqlen=1 if form == "step" else _log_int(rng, 2, 8192),
                 channels=groups * _log_int(rng, 16, 5120 // groups),
                 dstate=rng.choice((8, 16, 16, 16, 24, 33, 64)), groups=groups, dtype=dtype,
                 gate=rng.random() < 0.7, ragged=form == "fwd" and rng.random() < 0.5)
        while c["batch"] * c["seqlen"] * c["channels"] * c["dstate"] > 3e8:
            if c["seqlen"] > 1:
                c["seqlen"] = max(2, c["seqlen"] // 2)
            else:
                c["batch"] = max(1, c["batch"] // 2)
        return c
    dstate = rng.choice((16, 32, 64, 64, 128, 128, 128, 256))
    return dict(op=op, form=rng.choice(("fwd", "train")), batch=_log_int(rng, 1, 16),
                seqlen=_log_int(rng, 1, 4096), groups=rng.choice((1, 1, 2, 4, 5, 8)),
                dstate=dstate, rotary=rng.choice((dstate, dstate, dstate // 2)), dtype=dtype,
                interleaved=rng.random() < 0.5, far=rng.random() < 0.3)


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device="cuda") * std + mean).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    def lengths(b, L):
        n = torch.randint(max(1, L // 4), L + 1, (b,), generator=gen, device="cuda")
        return n.to(torch.int32)

    t = _dtype(case)
    s = dict(case=dict(case))
    b, L = case["batch"], case["seqlen"]
    if case["op"] == "conv":
        D, W = case["channels"], case["width"]
        s["weight"] = uniform(-1 / math.sqrt(W), 1 / math.sqrt(W), D, W)
        s["bias"] = uniform(-0.5, 0.5, D)
        if case["form"] == "step":
            s["x"] = normal(b, D, dtype=t)
            s["state"] = normal(b, W - 1, D, dtype=t)
            return s
        # the convolution's input is a view of the wider projection of the tokens
        s["x"] = normal(b, L, D + 256, dtype=t)[:, :, 64:64 + D]
        s["lens"] = lengths(b, L) if case["ragged"] else None
        if case["form"] == "train":
            s["dy"] = normal(b, L, D, dtype=t)
        return s
    if case["op"] == "scan":
        D, N, G = case["channels"], case["dstate"], case["groups"]
        s["A"] = -torch.arange(1, N + 1, device="cuda") * torch.exp(normal(D, N, std=0.1))
        s["D"] = normal(D, mean=1.0, std=0.1)
        step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), D))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))     # softplus(dt_bias) = step
        if case["form"] == "step":
            s["x"] = normal(b, D, dtype=t)
            s["dt"] = normal(b, D, std=0.5, dtype=t)
            s["B"], s["C"] = normal(b, G, N, dtype=t), normal(b, G, N, dtype=t)
            s["z"] = normal(b, D, dtype=t) if case["gate"] else None
            s["state"] = normal(b, D, N, std=0.1)
            return s
        s["x"] = normal(b, L, D, dtype=t)
        s["dt"] = normal(b, L, D, std=0.5, dtype=t)
        bc = normal(b, L, 2 * G * N, dtype=t)    # B and C are views of one projection
        s["B"], s["C"] = bc[:, :, :G * N].unflatten(2, (G, N)), bc[:, :, G * N:].unflatten(2, (G, N))
        # the gate is the other half of the projection that the convolution's input comes from
        s["z"] = normal(b, L, 2 * D, dtype=t)[:, :, D:] if case["gate"] else None
        s["lens"] = lengths(b, L) if case["ragged"] else None
        if case["form"] == "train":
            s["dy"] = normal(b, L, D, dtype=t)
            s["init"] = None if case["gate"] else normal(b, D, N, std=0.1)
        return s
    G, N, R = case["groups"], case["dstate"], case["rotary"]
    # B and C are views of the convolution's output, behind its other channels
    xbc = normal(b, L, 64 + 2 * G * N, dtype=t)[:, :, 64:]
    s["B"], s["C"] = xbc[:, :, :G * N].unflatten(2, (G, N)), xbc[:, :, G * N:].unflatten(2, (G, N))
    s["wB"], s["wC"] = normal(G, N, mean=1.0, std=0.1), normal(G, N, mean=1.0, std=0.1)
    start = torch.randint(0, 1 << 20, (b, 1), generator=gen, device="cuda") if case["far"] else 0
    s["pos"] = (torch.arange(L, device="cuda")[None, :] + start).expand(b, L).contiguous()
    s["freq"] = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float32) / R)
    if case["form"] == "train":
        s["dB"], s["dC"] = normal(b, L, G, N), normal(b, L, G, N)    # the scan's gradients: fp32
    return s


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    b, L, train = case["batch"], case["seqlen"], case["form"] == "train"
    if case["op"] == "conv":
        D, W = case["channels"], case["width"]
        n = b * L * D
        if case["form"] == "step":
            return {"bytes": n * e * (2 + 2 * (W - 1)) + 4 * D * (W + 1), "flops": n * (2 * W + 6)}
        return {"bytes": n * e * (4 if train else 2) + 4 * D * (W + 1) * (2 if train else 1),
                "flops": n * (2 * W + 6) * (3 if train else 1)}
    if case["op"] == "scan":
        D, N, G = case["channels"], case["dstate"], case["groups"]
        n, bc, z = b * L * D, 2 * b * L * G * N * e, 1 if case["gate"] else 0
        par, state = 4 * D * (N + 2), 4 * b * D * N
        if case["form"] == "step":
            return {"bytes": n * e * (3 + z) + bc + par + 2 * state, "flops": n * (8 * N + 12)}
        if train:   # x, dt, z, dy in; y, dx, ddt, dz out
            return {"bytes": n * e * (6 + 2 * z) + 2 * bc + 2 * par + (0 if z else 2 * state),
                    "flops": n * (28 * N + 40)}
        return {"bytes": n * e * (3 + z) + bc + par + state, "flops": n * (8 * N + 12)}
    G, N = case["groups"], case["dstate"]
    n = 2 * b * L * G * N
    if train:       # B, C and their fp32 gradients in; B, C and the gradients out
        return {"bytes": n * (3 * e + 4) + 8 * b * L + 16 * G * N, "flops": n * 20}
    return {"bytes": n * 2 * e + 8 * b * L + 8 * G * N, "flops": n * 8}


# ------------------------------------------------------------------ the plain forms
def _silu_slope(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def _inside(lens, b, L, device):
    """(b, L, 1): whether a token is one of its sequence's own."""
    at = torch.arange(L, device=device)[None, :, None]
    return at < (lens[:, None, None] if lens is not None else torch.full((b, 1, 1), L, device=device))


def _plain_conv(s):
    x, w = s["x"].float(), s["weight"]
    b, L, D = x.shape
    W = w.shape[1]
    inside = _inside(s["lens"], b, L, x.device)
    padded = torch.cat((x.new_zeros(b, W - 1, D), x), 1)
    window = padded.unfold(1, W, 1)                        # (b, L, D, W)
    pre = (window * w).sum(-1) + s["bias"]
    y = (pre * torch.sigmoid(pre) * inside).to(s["x"].dtype)
    if "dy" not in s:
        n = s["lens"].long() if s["lens"] is not None else torch.full((b,), L, device=x.device)
        at = n[:, None] + torch.arange(W - 1, device=x.device)
        state = padded.gather(1, at[:, :, None].expand(b, W - 1, D))
        return {"y": y, "state": state.to(s["x"].dtype)}
    g = s["dy"].float() * _silu_slope(pre)
    after = torch.cat((g, g.new_zeros(b, W - 1, D)), 1).unfold(1, W, 1)
    return {"y": y, "dx": (after * w.flip(1)).sum(-1).to(s["x"].dtype),
            "dweight": (g[..., None] * window).sum((0, 1)), "dbias": g.sum((0, 1))}


def _plain_conv_token(s):
    window = torch.cat((s["state"], s["x"][:, None]), 1)
    pre = (window.float() * s["weight"].t()).sum(1) + s["bias"]
    s["state"].copy_(window[:, 1:])
    return {"y": (pre * torch.sigmoid(pre)).to(s["x"].dtype), "state": s["state"]}


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension 1, from zero: pairs of tokens are
    joined, the half as long sequence is solved, and its states are spread."""
    L = u.shape[1]
    if L == 1:
        return u
    if L % 2:
        h = _linear_scan(a[:, :-1], u[:, :-1])
        return torch.cat((h, a[:, -1:] * h[:, -1:] + u[:, -1:]), 1)
    a0, a1, u0, u1 = a[:, 0::2], a[:, 1::2], u[:, 0::2], u[:, 1::2]
    odd = _linear_scan(a0 * a1, a1 * u0 + u1)
    even = u0.clone()
    even[:, 1:] += a0[:, 1:] * odd[:, :-1]
    return torch.stack((even, odd), 2).flatten(1, 2)


def _softplus(v):
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(s):
    """Channels as (G, D / G): B and C of a group serve its channels."""
    x = s["x"].float()
    b, L, D = x.shape
    G, N = s["B"].shape[2:]
    split = lambda v: v.unflatten(-1, (G, D // G))                      # noqa: E731
    inside = _inside(s["lens"], b, L, x.device)
    raw = s["dt"].float() + s["dt_bias"]
    dt = split(_softplus(raw) * inside)
    xs, A, Dv = split(x), s["A"].unflatten(0, (G, D // G)), split(s["D"])
    Bm, Cm = s["B"].float()[:, :, :, None], s["C"].float()[:, :, :, None]
    a = torch.exp(dt[..., None] * A)
    u = (dt * xs)[..., None] * Bm
    init = s.get("init")
    h0 = init.unflatten(1, (G, D // G)) if init is not None else None
    if h0 is not None:
        u[:, 0] += a[:, 0] * h0
    h = _linear_scan(a, u)
    del u
    core = (h * Cm).sum(-1) + Dv * xs
    z = s["z"].float() if s["z"] is not None else None
    gate = split(z * torch.sigmoid(z)) if z is not None else torch.ones_like(core)
    y = ((core * gate).flatten(2) * inside).to(s["x"].dtype)
    if "dy" not in s:
        return {"y": y, "state": h[:, -1].flatten(1, 2).contiguous()}
    dy = split(s["dy"].float())
    dyg = dy * gate
    after = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1).flip(1)
    g = _linear_scan(after, (dyg[..., None] * Cm).flip(1)).flip(1)
    del after
    low = s["x"].dtype
    out = {"y": y, "dC": (dyg[..., None] * h).sum(3).to(low),
           "dB": ((dt * xs)[..., None] * g).sum(3).to(low), "dD": (dyg * xs).sum((0, 1)).flatten()}
    du = (g * Bm).sum(-1)
    before = torch.cat((h0[:, None] if h0 is not None else torch.zeros_like(h[:, :1]), h[:, :-1]), 1)
    del h
    q = g * a * before
    if h0 is not None:
        out["dinit"] = (a[:, 0] * g[:, 0]).flatten(1, 2)
    del a, g, before
    ddt = ((q * A).sum(-1) + du * xs).flatten(2) * torch.sigmoid(raw)
    out["dA"] = (q * dt[..., None]).sum((0, 1)).flatten(0, 1)
    out["ddt"], out["ddt_bias"] = ddt.to(low), ddt.sum((0, 1))
    out["dx"] = (du * dt + dyg * Dv).flatten(2).to(low)
    if z is not None:
        out["dz"] = ((dy * core).flatten(2) * _silu_slope(z)).to(low)
    return out


def _plain_scan_token(s):
    x = s["x"].float()
    b, D = x.shape
    G, N = s["B"].shape[1:]
    per = lambda v: v.float().repeat_interleave(D // G, 1)              # noqa: E731
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(dt[..., None] * s["A"]) * s["state"] + (dt * x)[..., None] * per(s["B"])
    s["state"].copy_(h)
    y = (h * per(s["C"])).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


def _turn(v, angle, interleaved, back=False):
    """The first 2 * angle.shape[-1] elements of each row, in pairs, by their angles."""
    R = 2 * angle.shape[-1]
    cos, sin = angle.cos().to(v.dtype)[:, :, None], angle.sin().to(v.dtype)[:, :, None]
    sin = -sin if back else sin
    p, q = (v[..., 0:R:2], v[..., 1:R:2]) if interleaved else (v[..., :R // 2], v[..., R // 2:R])
    p, q = p * cos - q * sin, p * sin + q * cos
    turned = torch.stack((p, q), -1).flatten(-2) if interleaved else torch.cat((p, q), -1)
    return torch.cat((turned, v[..., R:]), -1)


def _plain_rotate(s):
    way = s["case"]["interleaved"]
    low = s["B"].dtype
    angle = s["pos"].double()[..., None] * s["freq"].double()
    B, C = s["B"].float(), s["C"].float()
    rB = torch.rsqrt((B * B).mean(-1, keepdim=True) + EPS)
    rC = torch.rsqrt((C * C).mean(-1, keepdim=True) + EPS)
    out = {"B": _turn(B * rB * s["wB"], angle, way).to(low),
           "C": _turn(C * rC * s["wC"], angle, way).to(low)}
    if "dB" in s:
        gB, gC = _turn(s["dB"], angle, way, True), _turn(s["dC"], angle, way, True)
        out["dwB"], out["dwC"] = (gB * B * rB).sum((0, 1)), (gC * C * rC).sum((0, 1))
        gB, gC = gB * s["wB"], gC * s["wC"]
        out["dB"] = (rB * (gB - B * rB * rB * (gB * B).mean(-1, keepdim=True))).to(low)
        out["dC"] = (rC * (gC - C * rC * rC * (gC * C).mean(-1, keepdim=True))).to(low)
    return out


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from ssd_chunked_scan_02_b200 import ssd
    case = s["case"]
    if case["op"] == "conv":
        if case["form"] == "step":
            y = ssd.ssd_causal_conv_step(s["state"], s["x"], s["weight"], s["bias"])
            return {"y": y, "state": s["state"]}
        if case["form"] == "fwd":
            y, state = ssd.ssd_causal_conv_fwd(s["x"], s["weight"], s["bias"], seq_lens=s["lens"],
                                               return_final_state=True)
            return {"y": y, "state": state}
        y = ssd.ssd_causal_conv_fwd(s["x"], s["weight"], s["bias"])
        g = ssd.ssd_causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], want_dinit=False)
        return {"y": y, "dx": g["dx"], "dweight": g["dweight"], "dbias": g["dbias"]}
    if case["op"] == "scan":
        more = dict(z=s["z"], dt_bias=s["dt_bias"], softplus=True)
        if case["form"] == "step":
            y = ssd.ssd_selective_step(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"],
                                       **more)
            return {"y": y, "state": s["state"]}
        if case["form"] == "fwd":
            y, state = ssd.ssd_selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"],
                                                  seq_lens=s["lens"], return_final_states=True,
                                                  **more)
            return {"y": y, "state": state}
        more["init_states"] = s["init"]
        y = ssd.ssd_selective_scan_fwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], **more)
        g = ssd.ssd_selective_scan_bwd(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dy"],
                                       want_dinit=s["init"] is not None, **more)
        return {"y": y, **{k: v for k, v in g.items() if v is not None}}
    args = (s["B"], s["C"], s["wB"], s["wC"], s["pos"], s["freq"])
    more = dict(eps=EPS, interleaved=case["interleaved"])
    B, C = ssd.ssd_bc_norm_rotate_fwd(*args, **more)
    if case["form"] == "fwd":
        return {"B": B, "C": C}
    return {"B": B, "C": C, **ssd.ssd_bc_norm_rotate_bwd(*args, s["dB"], s["dC"], **more)}


def run(state):
    if own:
        return _own(state)
    op, token = state["case"]["op"], state["case"]["form"] == "step"
    if op == "conv":
        return _plain_conv_token(state) if token else _plain_conv(state)
    if op == "scan":
        return _plain_scan_token(state) if token else _plain_scan(state)
    return _plain_rotate(state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_conv(s):
    x, w, bias = s["x"].double(), s["weight"].double(), s["bias"].double()
    if "state" in s:
        rows = list(s["state"].double().unbind(1)) + [x]
        pre = bias + sum(r * w[:, k] for k, r in enumerate(rows))
        return {"y": pre / (1 + torch.exp(-pre)), "state": torch.stack(rows[1:], 1)}
    b, L, D = x.shape
    W = w.shape[1]
    pre = bias.expand(b, L, D).clone()
    for k in range(W):              # tap k reads the token W - 1 - k before
        back = W - 1 - k
        if back < L:
            pre[:, back:] += x[:, :L - back] * w[:, k]
    sig = 1 / (1 + torch.exp(-pre))
    y = pre * sig
    if "dy" not in s:
        n = [int(v) for v in s["lens"]] if s["lens"] is not None else [L] * b
        state = x.new_zeros(b, W - 1, D)
        for i in range(b):
            y[i, n[i]:] = 0
            kept = min(W - 1, n[i])
            if kept:
                state[i, W - 1 - kept:] = x[i, n[i] - kept:n[i]]
        return {"y": y, "state": state}
    g = s["dy"].double() * (sig + y * (1 - sig))
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    for k in range(W):
        back = W - 1 - k
        if back < L:
            dx[:, :L - back] += g[:, back:] * w[:, k]
            dw[:, k] = (g[:, back:] * x[:, :L - back]).sum((0, 1))
    return {"y": y, "dx": dx, "dweight": dw, "dbias": g.sum((0, 1))}


def _exact_scan(s):
    """The recurrence token by token, its reverse likewise."""
    token = "state" in s
    up = lambda v: v.double()[:, None] if token else v.double()         # noqa: E731
    x, raw = up(s["x"]), up(s["dt"]) + s["dt_bias"].double()
    b, L, D = x.shape
    Bm, Cm = up(s["B"]), up(s["C"])
    G = Bm.shape[2]
    group = torch.arange(D, device=x.device) // (D // G)
    A, Dv = s["A"].double(), s["D"].double()
    dt = torch.where(raw > 30, raw, torch.log1p(torch.exp(raw)))
    lens = s.get("lens")
    z = up(s["z"]) if s["z"] is not None else None
    sig = 1 / (1 + torch.exp(-z)) if z is not None else None
    train = "dy" in s
    h = s["state"].double() if token else s["init"].double() if s.get("init") is not None else \
        x.new_zeros(b, D, A.shape[1])
    y, states = torch.empty_like(x), [h]
    for t in range(L):
        nxt = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * x[:, t])[..., None] * Bm[:, t, group]
        h = torch.where((t < lens)[:, None, None], nxt, h) if lens is not None else nxt
        y[:, t] = torch.einsum("bdn,bdn->bd", h, Cm[:, t, group]) + Dv * x[:, t]
        if train:
            states.append(h)
    if not train:
        out = y * z * sig if z is not None else y
        if lens is not None:
            out = out * (torch.arange(L, device=x.device)[None, :] < lens[:, None])[..., None]
        return {"y": out[:, 0] if token else out, "state": h}
    dy = s["dy"].double()
    dyg = dy * z * sig if z is not None else dy
    dx, ddt = torch.empty_like(x), torch.empty_like(x)
    dB, dC = torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA, g = torch.zeros_like(A), torch.zeros_like(h)
    for t in range(L - 1, -1, -1):
        g = g + dyg[:, t, :, None] * Cm[:, t, group]          # dL/dh_t
        a = torch.exp(dt[:, t, :, None] * A)
        dC[:, t].index_add_(1, group, dyg[:, t, :, None] * states[t + 1])
        dB[:, t].index_add_(1, group, (dt[:, t] * x[:, t])[..., None] * g)
        du = torch.einsum("bdn,bdn->bd", g, Bm[:, t, group])
        q = g * a * states[t]
        ddt[:, t] = torch.einsum("bdn,dn->bd", q, A) + du * x[:, t]
        dA += torch.einsum("bdn,bd->dn", q, dt[:, t])
        dx[:, t] = du * dt[:, t] + dyg[:, t] * Dv
        g = a * g
    draw_ = ddt / (1 + torch.exp(-raw))
    out = {"y": y * z * sig if z is not None else y, "dx": dx, "ddt": draw_, "dA": dA, "dB": dB,
           "dC": dC, "dD": (dyg * x).sum((0, 1)), "ddt_bias": draw_.sum((0, 1))}
    if z is not None:
        out["dz"] = dy * y * (sig + z * sig * (1 - sig))
    if s["init"] is not None:
        out["dinit"] = g
    return out


def _exact_rotate(s):
    """Each pair as a complex number, turned by exp(i pos freq)."""
    R, way = 2 * s["freq"].numel(), s["case"]["interleaved"]
    phase = s["pos"].double()[..., None] * s["freq"].double()
    turn = torch.polar(torch.ones_like(phase), phase)[:, :, None]
    N = s["B"].shape[-1]
    i = torch.arange(R // 2, device=phase.device)
    first, second = (2 * i, 2 * i + 1) if way else (i, i + R // 2)

    def rotated(v, by):
        c = torch.complex(v[..., first], v[..., second]) * by
        out = v.clone()
        out[..., first], out[..., second] = c.real, c.imag
        return out

    out = {}
    for k in ("B", "C"):
        v, w = s[k].double(), s["w" + k].double()
        root = torch.sqrt(v.square().sum(-1, keepdim=True) / N + EPS)
        out[k] = rotated(v / root * w, turn)
        if "dB" in s:
            g = rotated(s["d" + k].double(), turn.conj())
            out["dw" + k] = (g * v / root).sum((0, 1))
            g = g * w
            out["d" + k] = g / root - v * (g * v).sum(-1, keepdim=True) / (N * root ** 3)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "rotate": _exact_rotate}[case["op"]](s)
