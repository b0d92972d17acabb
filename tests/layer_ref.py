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
