"""The operators around the layer in a row, as a model runs them, in fp32 against
their fp64 definitions: convolution -> norm and rotation of B and C -> the SSD
layer, forward, gradients and single tokens behind a prompt; and convolution ->
selective scan with its gate, prompts of different lengths in one batch, then
single tokens from a captured graph.

Bounds.  Every operator here is off by a few 2^-24 of its terms and the SSD
layer by its own bound, 1e-4 of the largest element of a result (TOL["f32"]); the
operators before and behind it change that by factors of order one (norms of
weight one, convolutions whose weights' absolute values add up to about one), so
that the whole path is held to twice that bound."""
import pytest
import torch

import layer_ref as R
from parity import TOL, rel_err
from ssd_chunked_scan_02_b200 import build as ssd_build
from ssd_chunked_scan_02_b200 import ssd

BOUND = 2 * TOL["f32"]
EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


def close(name, got, ref):
    err = rel_err(R.f64(got).numpy(), ref.detach().numpy())
    assert err <= BOUND, (name, err)


H, P, N, G, W = 4, 16, 16, 2, 4
INNER, CH = H * P, H * P + 2 * G * N


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)                              # noqa: E731
    p = dict(conv_w=n(CH, W) * 0.3, conv_b=n(CH) * 0.1, A=-torch.rand(H, generator=g) * 8 - 0.5,
             D=n(H), wB=1 + 0.1 * n(G, N), wC=1 + 0.1 * n(G, N),
             freq=10000.0 ** (-torch.arange(0, N, 2) / N))
    return p, g


def ref_ssd(x, dt, A, B, C, D, h):
    """(y, state), the layer's recurrence: h <- exp(dt A) h + dt x B, y = C h + D x."""
    of = torch.arange(H) // (H // G)
    ys = []
    for t in range(x.shape[1]):
        h = torch.exp(dt[:, t] * A)[..., None, None] * h + \
            (dt[:, t, :, None] * x[:, t])[..., None] * B[:, t, of][:, :, None]
        ys.append((h * C[:, t, of][:, :, None]).sum(-1) + D[:, None] * x[:, t])
    return torch.stack(ys, 1), h


def ref_path(xbc, dt, p, pos):
    """conv -> norm and rotation -> SSD layer, from zero states."""
    b, L = xbc.shape[:2]
    u, state = R.conv(xbc, p["conv_w"], p["conv_b"], None, None, True)
    x = u[..., :INNER].unflatten(2, (H, P))
    B = u[..., INNER:INNER + G * N].unflatten(2, (G, N))
    C = u[..., INNER + G * N:].unflatten(2, (G, N))
    B = R.norm_rotate(B, p["wB"], pos, p["freq"], EPS, False)
    C = R.norm_rotate(C, p["wC"], pos, p["freq"], EPS, False)
    y, h = ref_ssd(x, dt, p["A"], B, C, p["D"], xbc.new_zeros(b, H, P, N))
    return y, h, state


def conv_parts(xbc, p, **k):
    """The convolution of x's channels and of B's and C's, each dense."""
    c = slice(0, INNER), slice(INNER, CH)
    return [ssd.ssd_causal_conv_fwd(xbc[..., s], p["conv_w"][s], p["conv_b"][s], **k) for s in c]


def bc_of(u):
    return u[..., :G * N].unflatten(-1, (G, N)), u[..., G * N:].unflatten(-1, (G, N))


@pytest.mark.gpu
def test_ssd_path_prompt_and_tokens(lib):
    p, g = weights(1)
    b, L, k = 2, 150, 4
    wide = torch.randn(b, L + k, CH + 24, generator=g)     # the projection: gate, xBC, dt
    dt = torch.rand(b, L + k, H, generator=g) * 0.1 + 0.001
    pos = torch.arange(L + k).expand(b, -1).contiguous() + torch.tensor([[3], [70000]])
    ry, rh, rs = ref_path(R.f64(wide[..., 16:16 + CH]), dt.double(), {k_: v.double() for k_, v in p.items()}, pos)
    p = {k_: v.cuda() for k_, v in p.items()}
    xbc, dt, pos = wide.cuda()[..., 16:16 + CH], dt.cuda(), pos.cuda()

    (x, sx), (u, su) = conv_parts(xbc[:, :L], p, return_final_state=True)
    B, C = ssd.ssd_bc_norm_rotate_fwd(*bc_of(u), p["wB"], p["wC"], pos[:, :L].contiguous(), p["freq"],
                                      eps=EPS)
    y, h = ssd.ssd_chunk_scan_fwd(x.unflatten(2, (H, P)), dt[:, :L].contiguous(), p["A"], B, C, p["D"],
                                  64, return_final_states=True)
    close("prompt", y, ry[:, :L])
    for t in range(L, L + k):
        x = ssd.ssd_causal_conv_step(sx, xbc[:, t, :INNER], p["conv_w"][:INNER], p["conv_b"][:INNER])
        u = ssd.ssd_causal_conv_step(su, xbc[:, t, INNER:], p["conv_w"][INNER:], p["conv_b"][INNER:])
        B, C = ssd.ssd_bc_norm_rotate_fwd(*bc_of(u[:, None]), p["wB"], p["wC"],
                                          pos[:, t:t + 1].contiguous(), p["freq"], eps=EPS)
        y = ssd.ssd_step(h, x.unflatten(1, (H, P)), dt[:, t].contiguous(), p["A"], B[:, 0].contiguous(),
                         C[:, 0].contiguous(), p["D"])
        close(f"token {t}", y, ry[:, t])
    close("state", h, rh)
    assert torch.equal(R.f64(torch.cat((sx, su), 2)), rs)


@pytest.mark.gpu
def test_ssd_path_gradients(lib):
    """The gradients' chain: the layer's fp32 gradients of B and C go into the norm
    and rotation as they are."""
    p, g = weights(2)
    b, L = 2, 90
    xbc, dt = torch.randn(b, L, CH, generator=g), torch.rand(b, L, H, generator=g) * 0.1 + 0.001
    pos = torch.arange(L).expand(b, -1).contiguous()
    dy = torch.randn(b, L, H, P, generator=g)
    leaf = {k: v.double().requires_grad_(k != "freq") for k, v in p.items()}
    lx, ld = xbc.double().requires_grad_(), dt.double().requires_grad_()
    y, _, _ = ref_path(lx, ld, leaf, pos)
    keys = ["conv_w", "conv_b", "A", "D", "wB", "wC"]
    ref = torch.autograd.grad((y * dy.double()).sum(), [lx, ld] + [leaf[k] for k in keys])
    ref = dict(zip(["xbc", "dt"] + keys, ref))

    p = {k: v.cuda() for k, v in p.items()}
    xbc, dt, pos, dy = xbc.cuda(), dt.cuda(), pos.cuda(), dy.cuda()
    x, u = conv_parts(xbc, p)
    B0, C0 = bc_of(u)
    more = (p["wB"], p["wC"], pos, p["freq"])
    B, C = ssd.ssd_bc_norm_rotate_fwd(B0, C0, *more, eps=EPS)
    s = ssd.ssd_chunk_scan_bwd(x.unflatten(2, (H, P)), dt, p["A"], B, C, p["D"], dy)
    r = ssd.ssd_bc_norm_rotate_bwd(B0, C0, *more, s["dB"], s["dC"], eps=EPS)
    du = torch.cat((r["dB"].flatten(2), r["dC"].flatten(2)), 2)
    gx = ssd.ssd_causal_conv_bwd(xbc[..., :INNER], p["conv_w"][:INNER], p["conv_b"][:INNER],
                                 s["dx"].flatten(2))
    gu = ssd.ssd_causal_conv_bwd(xbc[..., INNER:], p["conv_w"][INNER:], p["conv_b"][INNER:], du)
    close("xbc", torch.cat((gx["dx"], gu["dx"]), 2), ref["xbc"])
    close("dt", s["ddt"], ref["dt"])
    close("conv_w", torch.cat((gx["dweight"], gu["dweight"])), ref["conv_w"])
    close("conv_b", torch.cat((gx["dbias"], gu["dbias"])), ref["conv_b"])
    for k, v in (("A", s["dA"]), ("D", s["dD"]), ("wB", r["dwB"]), ("wC", r["dwC"])):
        close(k, v, ref[k])


@pytest.mark.gpu
def test_selective_path_ragged_prompts_then_tokens_from_a_graph(lib):
    """Prompts of 0, 1 and 70 tokens in one padded batch; then tokens of all three,
    from one captured graph whose states live on between replays."""
    g = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(s, generator=g)                              # noqa: E731
    D, S, lens, k = 48, 16, [70, 0, 1], 3
    b, L = len(lens), max(lens)
    p = dict(w=n(D, W) * 0.3, b=n(D) * 0.1, A=-torch.exp(torch.rand(D, S, generator=g) * 2.8),
             D=n(D), bias=n(D) - 4, proj=n(D, 2 * S) / D ** 0.5)
    xz, raw = n(b, L, 2 * D), n(b, L, D)
    tok_xz, tok_raw = n(k, b, 2 * D), n(k, b, D)

    def ref():
        q = {k_: v.double() for k_, v in p.items()}
        ys, fin = [], []
        for i, m in enumerate(lens):             # every sequence by itself, its tokens behind
            x = torch.cat((xz[i, :m], tok_xz[:, i]))[None].double()
            dt = torch.cat((raw[i, :m], tok_raw[:, i]))[None].double()
            u, _ = R.conv(x[..., :D], q["w"], q["b"], None, None, True)
            bc = u @ q["proj"]
            y, h = R.scan(u, dt, q["A"], bc[..., None, :S], bc[..., None, S:], q["D"], x[..., D:],
                          q["bias"])
            ys.append(y[0])
            fin.append(h[0])
        return ys, torch.stack(fin)

    ry, rh = ref()
    c = {k_: v.cuda() for k_, v in p.items()}
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    xz, raw = xz.cuda(), raw.cuda()
    u, conv = ssd.ssd_causal_conv_fwd(xz[..., :D], c["w"], c["b"], seq_lens=ln, return_final_state=True)
    torch.backends.cuda.matmul.allow_tf32 = False
    bc = (u @ c["proj"])[:, :, None]
    more = dict(D=c["D"], dt_bias=c["bias"])
    y, h = ssd.ssd_selective_scan_fwd(u, raw, c["A"], bc[..., :S], bc[..., S:], z=xz[..., D:],
                                      seq_lens=ln, return_final_states=True, **more)
    for i, m in enumerate(lens):
        if m:
            close(f"prompt {i}", y[i, :m], ry[i][:m])
        assert not y[i, m:].any()

    x_in, dt_in = tok_xz[0].cuda(), tok_raw[0].cuda()
    kept = conv.clone(), h.clone()

    def token():
        u = ssd.ssd_causal_conv_step(conv, x_in[:, :D], c["w"], c["b"])
        bc = (u @ c["proj"])[:, None]
        return ssd.ssd_selective_step(h, u, dt_in, c["A"], bc[..., :S], bc[..., S:], z=x_in[:, D:], **more)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()                                   # the library's first call, before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = token()
    conv.copy_(kept[0])
    h.copy_(kept[1])
    for t in range(k):
        x_in.copy_(tok_xz[t])
        dt_in.copy_(tok_raw[t])
        graph.replay()
        close(f"token {t}", out, torch.stack([ry[i][m + t] for i, m in enumerate(lens)]))
    close("states", h, rh)


@pytest.mark.gpu
def test_offsets_beyond_32_bits(lib):
    """A sequence of more than 2^31 elements: its last rows against a call on them
    alone (the convolution bit for bit; the scan's spans differ, so that its bf16
    results are one rounding apart at most, 2^-7 of the value with what fp32 adds:
    its few hundred roundings stay below 2^-14 of the largest element)."""
    L, D, cut = (1 << 20) + 8, 2056, 600
    assert L * D > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty(1, L, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    w, b = torch.randn(D, 4, device="cuda", generator=g), torch.randn(D, device="cuda", generator=g)
    y = ssd.ssd_causal_conv_fwd(x, w, b)
    part = ssd.ssd_causal_conv_fwd(x[:, L - cut:], w, b,
                                   init_state=x[:, L - cut - 3:L - cut].contiguous())
    assert torch.equal(y[:, L - cut:], part)
    del y

    A = -torch.rand(D, 16, device="cuda", generator=g) * 8
    bc = torch.randn(1, L, 1, 32, device="cuda", generator=g).bfloat16()
    args = lambda s: (x[:, s], x[:, s], A, bc[:, s, :, :16], bc[:, s, :, 16:])   # noqa: E731
    bias = torch.full((D,), -4.0, device="cuda")
    y, h = ssd.ssd_selective_scan_fwd(*args(slice(None)), dt_bias=bias, return_final_states=True)
    _, before = ssd.ssd_selective_scan_fwd(*args(slice(0, L - cut)), dt_bias=bias,
                                           return_final_states=True)
    part, hp = ssd.ssd_selective_scan_fwd(*args(slice(L - cut, None)), dt_bias=bias,
                                          init_states=before, return_final_states=True)
    whole, part = y[0, L - cut:].double(), part[0].double()
    assert ((whole - part).abs() <= 2.0 ** -7 * part.abs() + 2.0 ** -14 * part.abs().max()).all()
    assert float((h - hp).abs().max()) <= 2.0 ** -14 * float(hp.abs().max())
    del y, whole, part

    rows = x.view(1, -1)[:, :(1 << 31) + 4096].view(1, -1, 2, 64)     # more than 2^31 elements of B
    C, L = rows, rows.shape[1]
    pos = torch.arange(L, device="cuda")[None]
    freq = 10000.0 ** (-torch.arange(0, 64, 2, device="cuda") / 64)
    one = torch.ones(64, device="cuda")
    B1, C1 = ssd.ssd_bc_norm_rotate_fwd(rows, C, one, one, pos, freq)
    B2, C2 = ssd.ssd_bc_norm_rotate_fwd(rows[:, L - 100:], C[:, L - 100:], one, one,
                                        pos[:, L - 100:].contiguous(), freq)
    assert torch.equal(B1[:, L - 100:], B2) and torch.equal(C1[:, L - 100:], C2)
