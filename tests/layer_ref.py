"""Plain fp64 implementations of the operators around the layer, written token
by token from their definitions (include/ssd.h), and the comparison their
tests use.  Gradients come from autograd on these definitions."""
from __future__ import annotations

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # relative, one rounding
U = 2.0 ** -24                                                       # one fp32 rounding


def f64(t):
    return None if t is None else t.detach().double().cpu()


def own_lengths(lens, b, L):
    return [L] * b if lens is None else [min(max(int(n), 0), L) for n in lens]


def within(name, got, ref, bound):
    """|got - ref| <= one rounding to got's type + bound, element by element
    (bound: a tensor or a number; non-finite values have to be the same)."""
    got64, ref = f64(got), ref.detach().cpu().double()
    assert got64.shape == ref.shape, (name, got64.shape, ref.shape)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got64), torch.isnan(ref)), name
    inf = ~fine & ~torch.isnan(ref)
    assert torch.equal(got64[inf], ref[inf]), name
    tol = HALF_STEP[got.dtype] * 1.001 * ref.abs() + torch.as_tensor(bound, dtype=torch.float64)
    off = (got64 - ref).abs()
    bad = fine & (off > tol)
    if bad.any():
        i = int((off / tol).nan_to_num(0).flatten().argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} elements out of bounds; "
                             f"worst at {i}: got {got64.flatten()[i]:.9g}, want "
                             f"{ref.flatten()[i]:.9g}, bound {tol.expand_as(ref).flatten()[i]:.3g}")


# ------------------------------------------------------------------ causal convolution
def conv(x, w, bias, init, lens, silu):
    """(y, final state), fp64, differentiable."""
    b, L, D = x.shape
    W = w.shape[1]
    init = x.new_zeros(b, W - 1, D) if init is None else init
    ys, fs = [], []
    for i, n in enumerate(own_lengths(lens, b, L)):
        rows = torch.cat((init[i], x[i, :n]), 0)
        out = [x.new_zeros(0, D)]
        for t in range(n):
            p = (rows[t:t + W] * w.t()).sum(0)
            p = p if bias is None else p + bias
            out.append((p * torch.sigmoid(p) if silu else p)[None])
        ys.append(torch.cat(out + [x.new_zeros(L - n, D)], 0))
        fs.append(rows[n:n + W - 1])
    return torch.stack(ys), torch.stack(fs)


# ------------------------------------------------------------------ norm and rotation of B and C
def norm_rotate(v, w, pos, freq, eps, interleaved):
    """v (b,L,G,N), w (N) or (G,N), pos (b,L), freq (R/2): fp64, differentiable."""
    R = 2 * freq.numel()
    u = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * w
    f = (pos.double()[..., None] * freq.double())[:, :, None]
    c, s = torch.cos(f), torch.sin(f)
    out = list(u.unbind(-1))
    for p in range(R // 2):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + R // 2)
        out[i], out[j] = u[..., i] * c[..., p] - u[..., j] * s[..., p], \
            u[..., i] * s[..., p] + u[..., j] * c[..., p]
    return torch.stack(out, -1)


# ------------------------------------------------------------------ selective scan
def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, init=None, lens=None):
    """(y, final states), fp64, differentiable; the recurrence token by token."""
    b, L, ch = x.shape
    G, N = B.shape[2:]
    of = torch.arange(ch) // (ch // G)
    v = dt if dt_bias is None else dt + dt_bias
    if softplus:
        v = torch.logaddexp(v, torch.zeros_like(v))
    h = x.new_zeros(b, ch, N) if init is None else init
    own = torch.tensor(own_lengths(lens, b, L))
    ys = [x.new_zeros(b, 0, ch)]
    for t in range(L):
        on = (t < own)[:, None]
        nxt = torch.exp(v[:, t, :, None] * A) * h + (v[:, t] * x[:, t])[..., None] * B[:, t, of]
        h = torch.where(on[..., None], nxt, h)
        y = (h * C[:, t, of]).sum(-1)
        y = y if D is None else y + D * x[:, t]
        y = y if z is None else y * z[:, t] * torch.sigmoid(z[:, t])
        ys.append(torch.where(on, y, torch.zeros_like(y))[:, None])
    return torch.cat(ys, 1), h


def scan_bounds(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, init=None, lens=None,
                dy=None, dfinal=None):
    """How far fp32 arithmetic may take each result, running error bounds beside
    the recurrences (all values fp64, absolute values throughout, in units of
    one rounding 2^-24):
      dt: 8 of |dt| for the softplus (an exponential and a polynomial), and what
        rounding the bias sum (and with it the exponent) moves it by
      a = exp(dt A): its argument is off by (8 + 2) |dt A|, ex2 by 3
      h: E_t = a E_{t-1} + (13 + 10 |dt A|) a H_{t-1} + 16 |u B|, H the recurrence of |h|
      g: the same in reverse from dyg C, dyg off by 8 + |z| (the sigmoid's argument)
      sums over N states: 8 in a lane, 5 joins; over channels: 32 by shuffles and
      shared memory, then the blocks in turn; over tokens: 8, then the others in turn."""
    b, L, ch = x.shape
    G, N = B.shape[2:]
    of = torch.arange(ch) // (ch // G)
    own = torch.tensor(own_lengths(lens, b, L))
    on = (torch.arange(L)[None, :] < own[:, None])[..., None]
    raw = dt if dt_bias is None else dt + dt_bias
    v = torch.logaddexp(raw, torch.zeros_like(raw)) if softplus else raw
    # rounding the sum of dt and its bias moves softplus by at most slope * that
    dv = 8 * v.abs() + (dt.abs() + (0 if dt_bias is None else dt_bias.abs())) * \
        (torch.sigmoid(raw) if softplus else 1)
    v, dv = v * on, dv * on
    rel = (dv / v.abs().clamp(min=1e-30))[..., None]            # relative error of dt
    e = (v[..., None] * A.abs() * (rel + 2) + 5)                # ... of a, in roundings
    a = torch.exp(v[..., None] * A)
    uB = (v * x).abs()[..., None] * B[:, :, of].abs() * on[..., None]
    H = x.new_zeros(b, ch, N) if init is None else init.abs()
    E = torch.zeros_like(H)
    Hs, Es = [H], [E]
    for t in range(L):
        E = a[:, t] * E + (e[:, t] + 3) * a[:, t] * H + (rel[:, t] + 6) * uB[:, t]
        H = a[:, t] * H + uB[:, t]
        Hs.append(H)
        Es.append(E)
    Ca, Ba = C[:, :, of].abs() * on[..., None], B[:, :, of].abs() * on[..., None]
    Dx = x.abs() * (0 if D is None else D.abs())
    Hn, En = torch.stack(Hs[1:], 1) if L else H[:, None][:, :0], torch.stack(Es[1:], 1) if L else H[:, None][:, :0]
    core, ecore = (Ca * Hn).sum(-1) + Dx, (Ca * (En + 16 * Hn)).sum(-1) + 4 * Dx
    gate = z.abs() * torch.sigmoid(z) if z is not None else torch.ones_like(x)
    zr = 10 + z.abs() if z is not None else torch.ones_like(x)
    out = {"y": U * gate * (ecore + zr * core) * on, "final": U * E}
    if dy is None:
        return out
    dyg = dy.abs() * gate * on
    g = torch.zeros_like(H) if dfinal is None else dfinal.abs()
    eg = torch.zeros_like(H)
    res = {k: torch.zeros(b, L, ch, dtype=torch.float64) for k in ("dx", "ddt")}
    dB, dC = (torch.zeros(b, L, G, N, dtype=torch.float64) for _ in range(2))
    dA, seen, total = torch.zeros(ch, N, dtype=torch.float64), 0, L * b / 8 + 16
    blocks = 40 + ch / G / 4
    for t in range(L - 1, -1, -1):
        cg = Ca[:, t] * dyg[:, t, :, None]
        eg = eg + (zr[:, t, :, None] + 4) * cg + g
        g = g + cg
        m = dyg[:, t, :, None]
        dC[:, t].index_add_(1, of, m * (En[:, t] + (zr[:, t, :, None] + blocks) * Hn[:, t]))
        ua = (v[:, t] * x[:, t]).abs()[..., None]
        dB[:, t].index_add_(1, of, ua * (eg + (rel[:, t] + blocks) * g))
        du, edu = (Ba[:, t] * g).sum(-1), (Ba[:, t] * (eg + 16 * g)).sum(-1)
        aH = a[:, t] * Hs[t]
        eaH = a[:, t] * Es[t] + (e[:, t] + 2) * aH
        q, eq = g * aH, eg * aH + g * (eaH + 2 * aH)
        res["ddt"][:, t] = (A.abs() * (eq + 18 * q)).sum(-1) + (edu + 3 * du) * x[:, t].abs()
        big = (A.abs() * q).sum(-1) + du * x[:, t].abs()
        if softplus:
            s = torch.sigmoid(raw[:, t])
            res["ddt"][:, t] = s * res["ddt"][:, t] + big * s * (10 + 2 * raw[:, t].abs())
            big = big * s
        res.setdefault("big_ddt", torch.zeros(b, L, ch, dtype=torch.float64))[:, t] = big
        Da = 0 if D is None else D.abs()
        res["dx"][:, t] = v[:, t].abs() * (edu + 3 * du) + dv[:, t] * du + \
            dyg[:, t] * Da * (zr[:, t] + 4)
        dA += (v[:, t, :, None].abs() * (eq + (rel[:, t] + total) * q)).sum(0)
        eg = a[:, t] * eg + (e[:, t] + 2) * a[:, t] * g
        g = a[:, t] * g
    out |= {"dx": U * res["dx"] * on, "ddt": U * res["ddt"] * on, "dA": U * dA, "dB": U * dB,
            "dC": U * dC, "dinit": U * eg,
            "dD": U * ((zr + total) * dyg * x.abs()).sum((0, 1)),
            "ddt_bias": U * ((res["ddt"] + total * res.get("big_ddt", torch.zeros_like(x))) * on
                             ).sum((0, 1))}
    if z is not None:
        s = torch.sigmoid(z)
        slope = s * (1 + (z * (1 - s)).abs())
        out["dz"] = U * dy.abs() * slope * (ecore + (12 + 2 * z.abs()) * core) * on
    return out
