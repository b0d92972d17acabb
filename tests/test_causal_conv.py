"""The short causal convolution: refusals (no GPU), and the forward, the
gradients and the single-token form against the fp64 definition.

Bounds.  With S = |bias| + sum |w x| per output, p is a sum of W + 1 fp32
terms: off by at most (W + 1) roundings of S.  silu multiplies it by a sigmoid
of relative error below (|p| + 6) roundings (__expf and one fast division, and
the rounding of its argument), and its slope is at most 1.1: 32 roundings of S
cover both for |p| < 20.  Where S itself is below one, 32 * 2^-24 * S holds
likewise, as every term scales with p."""
import ctypes

import pytest
import torch

import layer_ref as R
from ssd_chunked_scan_02_b200 import build as ssd_build
from ssd_chunked_scan_02_b200 import ssd


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


P = 0x1000        # a plausible address that no rejected call touches
ST = ssd.ssd_stride_t(64, 8)


def _fwd(lib, dims, x=P, xs=ST, w=P, bias=P, init=None, lens=None, y=P, fin=None, dt=ssd.SSD_BF16):
    return lib.ssd_causal_conv_fwd(x, xs, w, bias, init, lens, 1, y, fin, dims, dt, None)


@pytest.mark.parametrize("dims,want", [
    ((-1, 8, 8, 4), 1), ((1, -8, 8, 4), 1), ((1, 8, 0, 4), 1), ((1, 8, 8, 1), 2), ((1, 8, 8, 5), 2),
    ((1 << 31, 8, 8, 4), 2), ((1, 1 << 31, 8, 4), 2), ((1, (1 << 31) - 9, 8, 4), 2), ((1, 8, 1 << 30, 4), 2),
    ((1 << 20, 1 << 20, 64, 4), 2)])
def test_sizes_refused(lib, dims, want):
    d = ssd.ssd_conv_dims_t(*dims)
    n = ctypes.c_size_t(7)
    assert _fwd(lib, d) == want
    assert lib.ssd_causal_conv_bwd_workspace_size(d, 1, n) == want and n.value == 7
    assert lib.ssd_last_error_detail() != b""


def test_pointers_refused(lib):
    d = ssd.ssd_conv_dims_t(1, 8, 8, 4)
    assert _fwd(lib, None) == 1 and _fwd(lib, d, xs=None) == 1
    assert _fwd(lib, d, x=None) == 1 and _fwd(lib, d, w=None) == 1 and _fwd(lib, d, y=None) == 1
    assert _fwd(lib, d, x=P + 1) == 1 and b"element" in lib.ssd_last_error_detail()
    for k in ("w", "bias", "init", "y", "fin"):
        assert _fwd(lib, d, **{k: P + 8}) == 1 and b"16-byte" in lib.ssd_last_error_detail(), k
    assert _fwd(lib, d, lens=P + 2) == 1
    assert _fwd(lib, d, dt=7) == 1
    for bad, want in ((ssd.ssd_stride_t(-1, 8), 1), (ssd.ssd_stride_t(64, -8), 1),
                      (ssd.ssd_stride_t(64, 1 << 31), 2)):
        assert _fwd(lib, d, xs=bad) == want
    assert lib.ssd_causal_conv_step(P, P, ssd.ssd_stride_t(-1, 0), P, P, 1, P, d, 1, None) == 1
    # an empty batch, and no tokens without a final state, launch nothing
    assert _fwd(lib, ssd.ssd_conv_dims_t(0, 8, 8, 4), x=None, w=None, y=None) == 0
    assert _fwd(lib, ssd.ssd_conv_dims_t(2, 0, 8, 4), x=None, w=None, y=None) == 0
    assert lib.ssd_causal_conv_step(None, P, ST, P, P, 1, P, d, 1, None) == 1
    assert lib.ssd_causal_conv_step(P, P, ST, P, P, 1, P, None, 1, None) == 1


def test_backward_refused(lib):
    d = ssd.ssd_conv_dims_t(2, 300, 10, 4)
    n = ctypes.c_size_t(0)
    assert lib.ssd_causal_conv_bwd_workspace_size(d, 1, n) == 0
    assert n.value == 2 * 2 * 10 * 5 * 4            # 2 sequences x 2 tiles of 256 tokens
    def call(dw=P, db=P, ws=P, nws=n.value, dy=P):
        return lib.ssd_causal_conv_bwd(P, ST, P, P, None, None, 1, dy, 0, None, P, dw, db, None, d,
                                       1, ws, nws, None)
    assert call(dw=None) == 1 and call(db=None) == 1 and call(dy=None) == 1
    assert call(nws=n.value - 1) == 1 and b"workspace" in lib.ssd_last_error_detail()
    assert call(ws=None) == 1


def test_binding_refuses(lib):
    x, w = torch.zeros(2, 5, 8), torch.zeros(8, 4)
    for bad in (dict(x=x[0]), dict(weight=w[:7]), dict(weight=w.double()), dict(bias=w[:, 0]),
                dict(init_state=x), dict(seq_lens=torch.zeros(2)), dict(y=x[:, :4]),
                dict(x=x.double()), dict(x=x.transpose(1, 2)), dict(x=x)):
        a = {"x": x, "weight": w, **bad}
        with pytest.raises((ValueError, TypeError)):
            ssd.ssd_causal_conv_fwd(a.pop("x"), a.pop("weight"), **a)
    with pytest.raises(ValueError):
        ssd.ssd_causal_conv_step(torch.zeros(2, 2, 8), x[:, 0], w)
    with pytest.raises(ValueError):
        ssd.ssd_causal_conv_bwd(x, w, None, x[:, 1:])


# ------------------------------------------------------------------ on the GPU
def make(b, L, D, W, dtype, seed, view=0, init=True, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)                          # noqa: E731
    x = n(b, L, D + view).to(dtype).to(dev)
    x = x[..., view // 2:view // 2 + D]
    return dict(x=x, w=(n(D, W) * 0.5).to(dev), bias=n(D).to(dev),
                init=n(b, W - 1, D).to(dtype).to(dev) if init else None, gen=g)


def sizes_of(d):
    """S of the bounds, per token, and of the entering rows."""
    x, w = R.f64(d["x"]).abs(), R.f64(d["w"]).abs()
    init = R.f64(d["init"])
    s, _ = R.conv(x, w, R.f64(d["bias"]).abs() if d["bias"] is not None else None,
                  init.abs() if init is not None else None, None, False)
    return s


CASES = [  # b, L, D, W, dtype, view, init, lens, silu
    (2, 37, 64, 4, "bf16", 0, True, None, True),
    (1, 1, 8, 4, "bf16", 0, False, None, True),
    (3, 2, 40, 3, "bf16", 16, True, [2, 0, 1], True),
    (4, 300, 136, 4, "bf16", 64, True, [300, 1, 0, 77], True),
    (2, 65, 33, 4, "bf16", 0, True, None, True),           # odd channels: one at a time
    (2, 65, 64, 4, "bf16", 3, False, [64, 70], True),      # an odd slice; a length over L
    (2, 520, 24, 2, "f32", 0, True, [257, 256], True),
    (1, 130, 21, 4, "f32", 2, True, None, False),
    (2, 40, 12, 3, "f32", 4, False, [-5, 3], True),        # a negative length: empty
    (2, 300, 33, 4, "bf16", 3, True, [300, 131], True),    # odd, several runs
    (2, 300, 33, 3, "f32", 1, True, [299, 64], True),
]
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])) + c[4])
def test_forward(lib, case):
    b, L, D, W, dt, view, init, lens, silu = case
    d = make(b, L, D, W, DT[dt], 100 + L, view, init)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    y, f = ssd.ssd_causal_conv_fwd(d["x"], d["w"], d["bias"], init_state=d["init"], seq_lens=ln,
                                   silu=silu, return_final_state=True)
    ry, rf = R.conv(R.f64(d["x"]), R.f64(d["w"]), R.f64(d["bias"]), R.f64(d["init"]), lens, silu)
    R.within("y", y, ry, 32 * R.U * sizes_of(d))
    assert torch.equal(R.f64(f), rf)


def grads(d, lens, silu, dy, df, keys=("x", "w", "bias", "init")):
    leaf = {k: R.f64(d[k]).requires_grad_() for k in keys if d[k] is not None}
    full = {k: leaf.get(k) for k in keys}
    y, f = R.conv(full["x"], full["w"], full["bias"], full["init"], lens, silu)
    loss = (y * R.f64(dy)).sum() + ((f * R.f64(df)).sum() if df is not None else 0)
    got = torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)
    return {k: (torch.zeros_like(v) if g is None else g) for (k, v), g in zip(leaf.items(), got)}


@pytest.mark.gpu
@pytest.mark.parametrize("dyt", ["same", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:4])) + c[4])
def test_gradients(lib, case, dyt):
    """|g| <= 1.1 |dy| (the slope of silu), its error 64 roundings of |dy| (1 + S);
    dx sums W of them, dweight and dbias all the tokens: 64 in a run, 4 runs,
    then the partial rows in eight columns."""
    b, L, D, W, dt, view, init, lens, silu = case
    d = make(b, L, D, W, DT[dt], 200 + L, view, init)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    dy = torch.randn(b, L, D, generator=d["gen"]).to(DT[dt] if dyt == "same" else torch.float32).cuda()
    df = torch.randn(b, W - 1, D, generator=d["gen"]).to(DT[dt]).cuda() if init else None
    g = ssd.ssd_causal_conv_bwd(d["x"], d["w"], d["bias"], dy, init_state=d["init"],
                                dfinal_state=df, seq_lens=ln, silu=silu, want_dinit=init)
    ref = grads(d, lens, silu, dy, df)
    S = sizes_of(d)
    big = R.f64(dy).abs() * (1 + S)                   # bounds |g| and, times 64 U, its error
    z = torch.zeros(b, W - 1, D, dtype=torch.float64)
    wa, xa = R.f64(d["w"]).abs(), R.f64(d["x"]).abs()
    ahead = torch.cat((big, z), 1)
    dxb = sum(wa[:, k] * ahead[:, W - 1 - k:W - 1 - k + L] for k in range(W))
    R.within("dx", g["dx"], ref["x"], 64 * R.U * (dxb + 8))
    rows = -(-L // 256) * b
    steps = 64 + 64 + 4 + rows / 8 + 8
    back = torch.cat((z if d["init"] is None else R.f64(d["init"]).abs(), xa), 1)
    dwb = torch.stack([(big * back[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)
    R.within("dweight", g["dweight"], ref["w"], steps * R.U * dwb)
    R.within("dbias", g["dbias"], ref["bias"], steps * R.U * big.sum((0, 1)))
    if init:
        # the entering rows get what the first W - 1 tokens (and the final state) send back
        head = torch.cat((z, big, z), 1)
        ib = sum(wa[:, k] * head[:, W - 1 - k:2 * (W - 1) - k] for k in range(W))
        R.within("dinit", g["dinit"], ref["init"], 64 * R.U * (ib + 8))


@pytest.mark.gpu
def test_gradients_against_differences(lib):
    """Central differences of the fp64 definition along random directions:
    their own error is h^2 times a third derivative of order one, 1e-8 of the
    directional derivative's scale at h = 1e-5; the gradients' error is bounded
    by sqrt(n) * 64 roundings of it."""
    d = make(2, 50, 24, 4, torch.float32, 5)
    dy = torch.randn(2, 50, 24, generator=d["gen"]).cuda()
    df = torch.randn(2, 3, 24, generator=d["gen"]).cuda()
    g = ssd.ssd_causal_conv_bwd(d["x"], d["w"], d["bias"], dy, init_state=d["init"], dfinal_state=df)
    base = [R.f64(d[k]) for k in ("x", "w", "bias", "init")]
    loss = lambda a: sum((o * R.f64(q)).sum() for o, q in                       # noqa: E731
                         zip(R.conv(*a, None, True), (dy, df)))
    for i, k in enumerate(("dx", "dweight", "dbias", "dinit")):
        v = torch.randn(base[i].shape, generator=d["gen"], dtype=torch.float64)
        h = 1e-5
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * v, base[i] - h * v
        want = float(loss(up) - loss(dn)) / (2 * h)
        got = float((R.f64(g[k]) * v).sum())
        scale = float((R.f64(g[k]) * v).abs().sum())
        assert abs(got - want) <= 1e-5 * scale, (k, got, want, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("b,D,W,dt,view", [(5, 64, 4, "bf16", 0), (1, 33, 4, "bf16", 0),
                                           (3, 40, 2, "f32", 7), (2, 20, 3, "bf16", 4)])
def test_tokens_continue_a_prompt(lib, b, D, W, dt, view):
    """A prompt, then single tokens: the same as the whole sequence at once, bit
    for bit (the taps are added in the same order)."""
    L, k = 9, 5
    d = make(b, L + k, D, W, DT[dt], 7, view)
    whole, fin = ssd.ssd_causal_conv_fwd(d["x"], d["w"], d["bias"], init_state=d["init"],
                                         return_final_state=True)
    y, state = ssd.ssd_causal_conv_fwd(d["x"][:, :L], d["w"], d["bias"], init_state=d["init"],
                                       return_final_state=True)
    assert torch.equal(y, whole[:, :L])
    for t in range(L, L + k):
        assert torch.equal(ssd.ssd_causal_conv_step(state, d["x"][:, t], d["w"], d["bias"]),
                           whole[:, t])
    assert torch.equal(state, fin)


@pytest.mark.gpu
def test_values_behind_the_sequences_are_never_read(lib):
    """NaN in the padding reaches nothing; outputs there are zero."""
    d = make(3, 40, 32, 4, torch.bfloat16, 9)
    lens = [40, 7, 0]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    x, dy = d["x"].clone(), torch.randn(3, 40, 32, generator=d["gen"]).bfloat16().cuda()
    for i, n in enumerate(lens):
        x[i, n:], dy[i, n:] = float("nan"), float("nan")
    y, f = ssd.ssd_causal_conv_fwd(x, d["w"], d["bias"], d["init"], ln, return_final_state=True)
    g = ssd.ssd_causal_conv_bwd(x, d["w"], d["bias"], dy, d["init"], seq_lens=ln)
    for v in (y, f, *g.values()):
        assert torch.isfinite(v.float()).all()
    for i, n in enumerate(lens):
        assert not y[i, n:].any() and not g["dx"][i, n:].any()


@pytest.mark.gpu
def test_no_tokens(lib):
    d = make(2, 0, 16, 4, torch.bfloat16, 3)
    y, f = ssd.ssd_causal_conv_fwd(d["x"], d["w"], d["bias"], d["init"], return_final_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(f, d["init"])
    df = torch.randn(2, 3, 16, generator=d["gen"]).bfloat16().cuda()
    g = ssd.ssd_causal_conv_bwd(d["x"], d["w"], d["bias"], y, d["init"], dfinal_state=df)
    assert torch.equal(g["dinit"], df) and not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.gpu
def test_streams_graphs_and_repeats(lib):
    """Another stream, a captured call replayed on changed inputs, and the same
    bits from every run."""
    d = make(2, 700, 64, 4, torch.bfloat16, 11)
    dy = torch.randn(2, 700, 64, generator=d["gen"]).bfloat16().cuda()
    call = lambda **k: (ssd.ssd_causal_conv_fwd(d["x"], d["w"], d["bias"], **k),       # noqa: E731
                        ssd.ssd_causal_conv_bwd(d["x"], d["w"], d["bias"], dy, **k))
    y, g = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        y2, g2 = call(stream=stream)
        side.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[k], g2[k]) for k in g if g[k] is not None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y3, g3 = call()
    d["x"].mul_(2)
    dy.mul_(-1)
    graph.replay()
    y4, g4 = call()
    torch.cuda.synchronize()
    assert torch.equal(y3, y4) and not torch.equal(y, y4)
    assert all(torch.equal(g3[k], g4[k]) for k in g if g[k] is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(4, 300, 136, 4, "bf16", 64, True, [300, 1, 0, 77], True),
                                  (2, 65, 33, 3, "f32", 1, True, None, True),
                                  (2, 40, 12, 2, "bf16", 0, False, None, False)],
                         ids=lambda c: "x".join(map(str, c[:4])) + c[4])
def test_without_bias(lib, case):
    """bias = None is a bias of zero, bit for bit, and dbias is written all the same;
    both against the definition (bounds: test_forward's and test_gradients')."""
    b, L, D, W, dt, view, init, lens, silu = case
    d = make(b, L, D, W, DT[dt], 300 + L, view, init)
    d["bias"] = None
    zero = torch.zeros(D, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda") if lens else None
    more = dict(init_state=d["init"], seq_lens=ln, silu=silu)
    y, f = ssd.ssd_causal_conv_fwd(d["x"], d["w"], **more, return_final_state=True)
    R.within("y", y, R.conv(R.f64(d["x"]), R.f64(d["w"]), None, R.f64(d["init"]), lens, silu)[0],
             32 * R.U * sizes_of(d))
    assert torch.equal(y, ssd.ssd_causal_conv_fwd(d["x"], d["w"], zero, **more))
    dy = torch.randn(b, L, D, generator=d["gen"]).to(DT[dt]).cuda()
    g = ssd.ssd_causal_conv_bwd(d["x"], d["w"], None, dy, **more)
    for k, v in ssd.ssd_causal_conv_bwd(d["x"], d["w"], zero, dy, **more).items():
        assert torch.equal(g[k], v), k
    ref = grads(d | dict(bias=zero), lens, silu, dy, None)
    big = R.f64(dy).abs() * (1 + sizes_of(d))
    steps = 64 + 64 + 4 + -(-L // 256) * b / 8 + 8
    R.within("dbias", g["dbias"], ref["bias"], steps * R.U * big.sum((0, 1)))
    token = torch.randn(b, D, generator=d["gen"]).to(DT[dt]).cuda()
    states = [f.clone(), f.clone()]
    ys = [ssd.ssd_causal_conv_step(s, token, d["w"], v, silu=silu) for s, v in zip(states, (None, zero))]
    assert torch.equal(*ys) and torch.equal(*states)
