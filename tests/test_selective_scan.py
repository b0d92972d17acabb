"""The selective scan: refusals (no GPU), and the forward, the gradients and the
single-token form against the fp64 recurrence, within running error bounds
(layer_ref.scan_bounds)."""
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


P = 0x1000
ST = ssd.ssd_selective_strides_t(*[64, 8] * 5)


@pytest.mark.parametrize("dims,want", [
    ((-1, 8, 8, 4, 1), 1), ((1, -8, 8, 4, 1), 1), ((1, 8, 0, 4, 1), 1), ((1, 8, 8, 0, 1), 1),
    ((1, 8, 8, 4, 0), 1), ((1, 8, 8, 4, 3), 1), ((1, 8, 8, 257, 1), 2), ((1 << 31, 8, 8, 4, 1), 2),
    ((1 << 20, 8, 1 << 20, 4, 1), 2), ((1, 1 << 31, 8, 4, 1), 2)])
def test_sizes_refused(lib, dims, want):
    d = ssd.ssd_selective_dims_t(*dims)
    n = ctypes.c_size_t(7)
    assert lib.ssd_selective_scan_fwd(P, P, P, P, P, P, P, P, 1, None, None, P, None, ST, d, 1, P,
                                      1 << 40, None) == want
    for f in (lib.ssd_selective_scan_fwd_workspace_size, lib.ssd_selective_scan_bwd_workspace_size):
        assert f(d, 1, n) == want and n.value == 7
    if dims[1] == 8:            # the step ignores seqlen
        assert lib.ssd_selective_step(*[P] * 9, 1, P, ST, d, 1, None) == want


def test_pointers_refused(lib):
    d = ssd.ssd_selective_dims_t(2, 300, 24, 16, 2)
    good = [P, P, P, P, P, P, P, P, 1, P, P, P, P, ST, d, 1, P, 1 << 40, None]
    for i, bad in [(0, None), (0, P + 1), (1, None), (1, P + 1), (2, None), (2, P + 4), (3, None),
                   (4, None), (4, P + 1), (5, P + 4), (6, P + 1), (7, P + 8), (9, P + 8), (10, P + 1),
                   (11, None), (11, P + 2), (12, P + 4), (13, None), (14, None), (15, 9)]:
        a = list(good)
        a[i] = bad
        assert lib.ssd_selective_scan_fwd(*a) == 1, i
    n = ctypes.c_size_t(0)
    assert lib.ssd_selective_scan_bwd_workspace_size(d, 1, n) == 0 and n.value > 0
    good = [P] * 8 + [1, P, P, P, P] + [P] * 9 + [ST, d, 1, P, n.value, None]
    for i, bad in [(0, None), (2, None), (11, None), (12, P + 4), (13, None), (14, P + 2), (15, None),
                   (16, None), (17, None), (18, P + 4), (19, None), (20, P + 4), (21, P + 8),
                   (22, None), (25, None), (26, n.value - 1)]:
        a = list(good)
        a[i] = bad
        assert lib.ssd_selective_scan_bwd(*a) == 1, i
    good = [P] * 9 + [1, P, ST, d, 1, None]
    for i, bad in [(0, None), (0, P + 4), (1, None), (3, None), (4, P + 1), (10, None), (11, None),
                   (12, None)]:
        a = list(good)
        a[i] = bad
        assert lib.ssd_selective_step(*a) == 1, i
    none = ssd.ssd_selective_dims_t(0, 300, 24, 16, 2)
    assert lib.ssd_selective_scan_fwd(*[None] * 8, 1, *[None] * 4, ST, none, 1, None, 0, None) == 0
    assert lib.ssd_selective_step(*[None] * 9, 1, None, ST, none, 1, None) == 0


def test_binding_refuses(lib):
    x, A, B = torch.zeros(2, 5, 8), torch.zeros(8, 4), torch.zeros(2, 5, 2, 4)
    for bad in (dict(x=x[0]), dict(dt=x[:, :4]), dict(A=A[:, :3]), dict(A=A.double()),
                dict(B=B[:, :, 0]), dict(C=B[..., :3]), dict(C=B.bfloat16()), dict(D=A),
                dict(z=x[:1]), dict(dt_bias=A[0]), dict(init_states=torch.zeros(2, 4, 8)),
                dict(seq_lens=torch.zeros(2, dtype=torch.int64)), dict(y=x.bfloat16()),
                dict(z=x.transpose(0, 2)), dict(x=x.half()), dict()):
        a = dict(x=x, dt=x, A=A, B=B, C=B)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            ssd.ssd_selective_scan_fwd(**a)
    with pytest.raises(ValueError):
        ssd.ssd_selective_scan_bwd(x, x, A, B, B, None, x[:, 1:])
    with pytest.raises(ValueError):
        ssd.ssd_selective_step(torch.zeros(2, 4, 8), x[:, 0], x[:, 0], A, B[:, 0], B[:, 0])


# ------------------------------------------------------------------ on the GPU
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    def __init__(self, b, L, ch, N, G=1, dt="bf16", gate=True, skip=True, bias=True, softplus=True,
                 init=True, lens=None, view=0):
        self.__dict__.update(locals())

    def __repr__(self):
        return f"{self.b}x{self.L}x{self.ch}x{self.N}g{self.G}{self.dt}"


CASES = [
    Case(2, 70, 64, 16),
    Case(1, 1, 32, 16, init=False),
    Case(3, 33, 40, 16, lens=[33, 0, 7], view=8),
    Case(2, 100, 96, 16, G=3, dt="f32", gate=False, lens=[101, 64]),
    Case(2, 45, 33, 16, view=3),                       # odd channels and slices
    Case(1, 64, 20, 5, G=2, dt="f32", skip=False, bias=False),
    Case(2, 40, 130, 8, gate=False),                   # 64 channels a block
    Case(2, 50, 48, 24, G=2, init=False),
    Case(1, 37, 24, 33, view=5),
    Case(2, 31, 16, 64, dt="f32"),
    Case(1, 29, 12, 100, softplus=False),
    Case(1, 20, 9, 256, dt="f32", lens=[13]),
    Case(2, 300, 8, 1, skip=False),
    Case(15, 19, 960, 16, init=False),                 # more blocks than 148 SMs hold at once
    Case(4, 37, 500, 5, G=125, dt="f32", lens=[37, 36, 0, 17]),
    Case(2, 145, 33, 16, dt="f32", view=3, lens=[140, 3]),   # odd slices, element by element
    Case(3, 67, 41, 24, dt="f32", view=1, gate=False),
]


def make(c, seed=0, dev="cuda"):
    g = torch.Generator().manual_seed(seed + c.L * 7 + c.N)
    n = lambda *s: torch.randn(s, generator=g)                          # noqa: E731

    def token(width):
        return n(c.b, c.L, width + c.view).to(DT[c.dt]).to(dev)[..., c.view:]

    A = -torch.exp(torch.rand(c.ch, c.N, generator=g) * 2.8)            # -1 .. -16
    dt = token(c.ch)
    if not c.softplus:
        dt = (dt.abs() * 0.05).to(DT[c.dt])
    d = dict(x=token(c.ch), dt=dt, A=A.to(dev), B=token(c.G * c.N).unflatten(2, (c.G, c.N)),
             C=token(c.G * c.N).unflatten(2, (c.G, c.N)), D=n(c.ch).to(dev) if c.skip else None,
             z=token(c.ch) if c.gate else None,
             dt_bias=(n(c.ch) - 3 * c.softplus).to(dev) if c.bias else None,
             softplus=c.softplus)
    if c.bias and not c.softplus:
        d["dt_bias"] = d["dt_bias"].abs() * 0.01
    more = dict(init=n(c.b, c.ch, c.N).to(dev) if c.init else None, lens=c.lens, gen=g,
                lens_t=torch.tensor(c.lens, dtype=torch.int32, device=dev) if c.lens else None)
    return d, more


def ref_args(d, m):
    out = {k: (R.f64(v) if torch.is_tensor(v) else v) for k, v in d.items()}
    return out | dict(init=R.f64(m["init"]), lens=m["lens"])


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=repr)
def test_forward(lib, c):
    d, m = make(c)
    y, f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], seq_lens=m["lens_t"],
                                      return_final_states=True)
    ra = ref_args(d, m)
    ry, rf = R.scan(**ra)
    bound = R.scan_bounds(**ra)
    R.within("y", y, ry, bound["y"])
    R.within("final", f, rf, bound["final"])


NAMES = dict(dx="x", ddt="dt", dA="A", dB="B", dC="C", dD="D", dz="z", ddt_bias="dt_bias",
             dinit="init")


@pytest.mark.gpu
@pytest.mark.parametrize("c", CASES, ids=repr)
def test_gradients(lib, c):
    d, m = make(c, 1000)
    dy = torch.randn(c.b, c.L, c.ch, generator=m["gen"]).to(DT[c.dt]).cuda()
    df = torch.randn(c.b, c.ch, c.N, generator=m["gen"]).cuda() if c.init else None
    g = ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"], dfinal_states=df,
                                   seq_lens=m["lens_t"], want_dinit=c.init)
    ra = ref_args(d, m)
    leaf = {k: v.requires_grad_() for k, v in ra.items() if torch.is_tensor(v)}
    y, f = R.scan(**ra)
    loss = (y * R.f64(dy)).sum() + ((f * R.f64(df)).sum() if df is not None else 0)
    ref = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)))
    plain = {k: (v.detach() if torch.is_tensor(v) else v) for k, v in ra.items()}
    bound = R.scan_bounds(**plain, dy=R.f64(dy), dfinal=R.f64(df))
    for k, of in NAMES.items():
        if of not in leaf:
            assert g[k] is None, k
            continue
        want = ref[of] if ref[of] is not None else torch.zeros_like(leaf[of])
        R.within(k, g[k], want, bound[k])


@pytest.mark.gpu
def test_gradients_against_differences(lib):
    """Central differences of the fp64 definition; see the convolution's test."""
    c = Case(2, 21, 12, 16, G=2, dt="f32")
    d, m = make(c, 77)
    dy = torch.randn(2, 21, 12, generator=m["gen"]).cuda()
    df = torch.randn(2, 12, 16, generator=m["gen"]).cuda()
    g = ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"], dfinal_states=df)
    base = ref_args(d, m)

    def loss(a):
        y, f = R.scan(**a)
        return float((y * R.f64(dy)).sum() + (f * R.f64(df)).sum())
    for k, of in NAMES.items():
        v = torch.randn(base[of].shape, generator=m["gen"], dtype=torch.float64)
        h = 1e-5
        want = (loss({**base, of: base[of] + h * v}) - loss({**base, of: base[of] - h * v})) / (2 * h)
        got = R.f64(g[k]) * v
        assert abs(float(got.sum()) - want) <= 1e-5 * float(got.abs().sum()), k


@pytest.mark.gpu
@pytest.mark.parametrize("c", [CASES[0], CASES[4], CASES[3], CASES[8], CASES[11], CASES[12]],
                         ids=repr)
def test_tokens_continue_a_prompt(lib, c):
    """A prompt, then single tokens, each against the fp64 recurrence from the
    state that the call was given."""
    c = Case(**{**{k: v for k, v in c.__dict__.items() if k != "self"}, "lens": None})
    d, m = make(c, 5)
    k = min(4, c.L - 1)
    cut = lambda s: {q: (v[:, s] if torch.is_tensor(v) and v.dim() >= 3 else v)       # noqa: E731
                     for q, v in d.items()}
    y, state = ssd.ssd_selective_scan_fwd(**cut(slice(0, c.L - k)), init_states=m["init"],
                                          return_final_states=True)
    whole, fin = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], return_final_states=True)
    assert torch.equal(y, whole[:, :c.L - k])
    for t in range(c.L - k, c.L):
        before = state.clone()
        one = ssd.ssd_selective_step(state, **cut(t))
        ra = {q: (R.f64(v) if torch.is_tensor(v) else v) for q, v in cut(slice(t, t + 1)).items()}
        ry, rf = R.scan(**ra, init=R.f64(before))
        bound = R.scan_bounds(**ra, init=R.f64(before))
        R.within("y", one[:, None], ry, bound["y"])
        R.within("state", state, rf, bound["final"])
    ra = ref_args(d, m)
    R.within("final", state, R.scan(**ra)[1], R.scan_bounds(**ra)["final"])


@pytest.mark.gpu
def test_values_behind_the_sequences_are_never_read(lib):
    c = Case(3, 50, 40, 16, lens=[50, 9, 0])
    d, m = make(c, 3)
    dy = torch.randn(3, 50, 40, generator=m["gen"]).bfloat16().cuda()
    for i, n in enumerate(c.lens):
        for k in ("x", "dt", "B", "C", "z"):
            d[k][i, n:] = float("nan")
        dy[i, n:] = float("nan")
    y, f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], seq_lens=m["lens_t"],
                                      return_final_states=True)
    g = ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"], seq_lens=m["lens_t"])
    for v in (y, f, *g.values()):
        assert torch.isfinite(v.float()).all()
    for i, n in enumerate(c.lens):
        for v in (y, g["dx"], g["ddt"], g["dz"], g["dB"], g["dC"]):
            assert not v[i, n:].any()
    assert torch.equal(f[2], m["init"][2])


@pytest.mark.gpu
def test_extreme_steps(lib):
    """Steps of zero (the state stays), steps so long that nothing of the state is
    left, and a softplus far on both sides."""
    c = Case(1, 40, 32, 16, dt="f32", bias=False)
    d, m = make(c, 8)
    d["dt"][:, 5] = -200.0
    d["dt"][:, 11] = 90.0
    d["dt"][:, 17] = 1e4
    y, f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], return_final_states=True)
    ra = ref_args(d, m)
    ry, rf = R.scan(**ra)
    b = R.scan_bounds(**ra)
    R.within("y", y, ry, b["y"] + 1e-37)
    R.within("final", f, rf, b["final"] + 1e-37)
    dy = torch.randn(1, 40, 32, generator=m["gen"]).cuda()
    assert all(torch.isfinite(v).all() for v in
               ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"]).values() if v is not None)


@pytest.mark.gpu
def test_no_tokens(lib):
    c = Case(2, 0, 16, 16)
    d, m = make(c)
    y, f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], return_final_states=True)
    assert y.shape == (2, 0, 16) and torch.equal(f, m["init"])
    df = torch.randn(2, 16, 16, generator=m["gen"]).cuda()
    g = ssd.ssd_selective_scan_bwd(**d, dy=y, init_states=m["init"], dfinal_states=df)
    assert torch.equal(g["dinit"], df)
    assert not any(g[k].any() for k in ("dA", "dD", "ddt_bias"))


@pytest.mark.gpu
def test_streams_graphs_and_repeats(lib):
    c = Case(2, 300, 96, 16, G=2)
    d, m = make(c, 4)
    dy = torch.randn(2, 300, 96, generator=m["gen"]).bfloat16().cuda()
    def call(**k):
        f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], return_final_states=True, **k)
        return [*f, *ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"], **k).values()]
    one = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    two = call(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    d["x"].mul_(2)
    d["dt"].mul_(-1)
    dy.mul_(-1)
    graph.replay()
    want = call()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and not torch.equal(one[0], kept[0])


SPANS = [  # long and narrow: the sequence is cut into spans, of both walks
    Case(1, 700, 40, 16, lens=[650]),
    Case(2, 333, 24, 16, G=2, dt="f32", lens=[333, 64]),
    Case(1, 520, 33, 24, view=3, init=False),
    Case(1, 300, 12, 100, dt="f32"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("c", SPANS, ids=repr)
def test_spans(lib, c):
    """Few channels and many tokens.  The sums of dt over a span add up to L
    roundings of their size, and a span's decay that many of its exponent: the
    running bounds' 10 |dt A| a token cover it.  (Lengths that end inside a span,
    at its border, and before the last one.)"""
    d, m = make(c, 31)
    dims = ssd.ssd_selective_dims_t(c.b, c.L, c.ch, c.N, c.G)
    assert ssd.ssd_selective_scan_fwd_workspace_size(dims, DT[c.dt]) > 0
    y, f = ssd.ssd_selective_scan_fwd(**d, init_states=m["init"], seq_lens=m["lens_t"],
                                      return_final_states=True)
    dy = torch.randn(c.b, c.L, c.ch, generator=m["gen"]).to(DT[c.dt]).cuda()
    df = torch.randn(c.b, c.ch, c.N, generator=m["gen"]).cuda() if c.init else None
    g = ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=m["init"], dfinal_states=df,
                                   seq_lens=m["lens_t"], want_dinit=c.init)
    ra = ref_args(d, m)
    leaf = {k: v.requires_grad_() for k, v in ra.items() if torch.is_tensor(v)}
    ry, rf = R.scan(**ra)
    loss = (ry * R.f64(dy)).sum() + ((rf * R.f64(df)).sum() if df is not None else 0)
    ref = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()), allow_unused=True)))
    plain = {k: (v.detach() if torch.is_tensor(v) else v) for k, v in ra.items()}
    bound = R.scan_bounds(**plain, dy=R.f64(dy), dfinal=R.f64(df))
    R.within("y", y, ry, bound["y"])
    R.within("final", f, rf, bound["final"])
    for k, of in NAMES.items():
        if of in leaf:
            want = ref[of] if ref[of] is not None else torch.zeros_like(leaf[of])
            R.within(k, g[k], want, bound[k])


@pytest.mark.gpu
@pytest.mark.parametrize("c", [CASES[2], CASES[3], CASES[8], Case(1, 700, 24, 16, lens=[650])], ids=repr)
def test_states_that_forget_at_once(lib, c):
    # exp(dt A) is 0 for A = -inf as for A = -1e30 (dt > 1e-28), also where the rows
    # behind a sequence have a step of zero: the same bits, nothing of it NaN
    d, m = make(c, 2000)
    some = torch.rand(c.ch, c.N, generator=m["gen"]).cuda() < 0.3
    dy = torch.randn(c.b, c.L, c.ch, generator=m["gen"]).to(DT[c.dt]).cuda()
    got = []
    for low in (-float("inf"), -1e30):
        e = d | dict(A=torch.where(some, low, d["A"]))
        y, f = ssd.ssd_selective_scan_fwd(**e, init_states=m["init"], seq_lens=m["lens_t"],
                                          return_final_states=True)
        g = ssd.ssd_selective_scan_bwd(**e, dy=dy, init_states=m["init"], seq_lens=m["lens_t"])
        t = {k: e[k] if e[k] is None or k in ("A", "D", "dt_bias") else e[k][:, 0]
             for k in ("x", "dt", "A", "B", "C", "D", "z", "dt_bias")}
        state = f.clone()
        yt = ssd.ssd_selective_step(state, **t)
        got.append([y, f, state, yt] + [v for _, v in sorted(g.items()) if v is not None])
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.gpu
def test_step_with_groups_beyond_32_bits(lib):
    """A group a channel, more than 2^31 elements of B and C a sequence: the last
    channels against a call on them alone, bit for bit."""
    D, N, cut = (1 << 23) + 24, 256, 40
    assert (D - 1) * N > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(2)
    n = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16).normal_(generator=g)   # noqa: E731
    bc, x, dt = n(1, D, N), n(1, D), n(1, D)
    A = torch.empty(D, N, device="cuda").uniform_(-8, -0.1, generator=g)
    state = torch.empty(1, D, N, device="cuda").normal_(generator=g)
    tail = state[:, -cut:].clone()
    y = ssd.ssd_selective_step(state, x, dt, A, bc, bc)
    part = ssd.ssd_selective_step(tail, x[:, -cut:], dt[:, -cut:], A[-cut:], bc[:, -cut:], bc[:, -cut:])
    assert torch.equal(y[:, -cut:], part) and torch.equal(state[:, -cut:], tail)


@pytest.mark.gpu
def test_growing_states_over_spans(lib):
    """A > 0 over a sequence that is cut into spans: a state (or a gradient) of zero
    stays zero through any growth, and a small one grows as far as it does token
    by token, also where the growth alone is beyond fp32."""
    c = Case(1, 700, 40, 16, dt="f32", gate=False, skip=False, bias=False, softplus=False, init=False)
    dims = ssd.ssd_selective_dims_t(c.b, c.L, c.ch, c.N, c.G)
    assert ssd.ssd_selective_scan_fwd_workspace_size(dims, torch.float32) > 0
    d, m = make(c, 41)
    d["A"] = torch.full_like(d["A"], 4.0)

    def forward(init=None):
        y, f = ssd.ssd_selective_scan_fwd(**d, init_states=init, return_final_states=True)
        ra = ref_args(d, m) | dict(init=R.f64(init))
        ry, rf = R.scan(**ra)
        bound = R.scan_bounds(**ra)
        assert torch.isfinite(ry).all() and torch.isfinite(rf).all()
        R.within("y", y, ry, bound["y"])
        R.within("final", f, rf, bound["final"])
    # exp(4 * 128) before the first input
    d["dt"] = torch.full_like(d["dt"], 1e-3)
    d["dt"][:, :128] = 1.0
    d["x"][:, :128] = 0
    forward()
    # exp(97) = 2^140 over the first 64 tokens, of 1e-30
    d["dt"][:, :128] = 1e-3
    d["dt"][:, :64] = 97 / 256
    forward(torch.full((1, c.ch, c.N), 1e-30, device="cuda"))
    # in reverse: exp(4 * 100) behind the last token that has a gradient
    d["dt"][:] = 1e-3
    d["dt"][:, 600:] = 1.0
    d["x"][:] = 0
    dy = torch.randn(1, c.L, c.ch, generator=m["gen"]).cuda()
    dy[:, 600:] = 0
    g = ssd.ssd_selective_scan_bwd(**d, dy=dy)
    ra = ref_args(d, m)
    leaf = {k: v.requires_grad_() for k, v in ra.items() if torch.is_tensor(v)}
    y, _ = R.scan(**ra)
    ref = dict(zip(leaf, torch.autograd.grad((y * R.f64(dy)).sum(), list(leaf.values()))))
    bound = R.scan_bounds(**{k: (v.detach() if torch.is_tensor(v) else v) for k, v in ra.items()},
                          dy=R.f64(dy))
    for k, of in NAMES.items():
        if of in leaf:
            R.within(k, g[k], ref[of], bound[k])


@pytest.mark.gpu
@pytest.mark.parametrize("c", [Case(3, 50, 40, 16, lens=[50, 0, 5]), Case(3, 37, 24, 33, dt="f32", lens=[37, 0, 6]),
                               Case(3, 700, 40, 16, dt="f32", lens=[650, 0, 70])], ids=repr)
def test_empty_sequences_with_any_entering_state(lib, c):
    """What enters an empty sequence (a place of the batch that nobody uses: any
    bits, NaN among them) leaves it again, and reaches no other result; a state
    that overflowed is not seen in the rows behind its sequence."""
    d, m = make(c, 51)
    dy = torch.randn(c.b, c.L, c.ch, generator=m["gen"]).to(DT[c.dt]).cuda()
    df = torch.randn(c.b, c.ch, c.N, generator=m["gen"]).cuda()

    def call(init, df):
        y, f = ssd.ssd_selective_scan_fwd(**d, init_states=init, seq_lens=m["lens_t"], return_final_states=True)
        return dict(y=y, f=f, **ssd.ssd_selective_scan_bwd(**d, dy=dy, init_states=init, dfinal_states=df,
                                                           seq_lens=m["lens_t"]))
    init, dead, want = m["init"].clone(), df.clone(), None
    init[1], dead[1] = 0, 0
    want = call(init, dead)
    init[1], dead[1] = float("nan"), float("nan")
    init[1, ::2], dead[1, 1::2] = float("inf"), -float("inf")
    got = call(init, dead)
    assert torch.equal(got["f"][1].nan_to_num(7.0), init[1].nan_to_num(7.0))
    assert torch.equal(got["dinit"][1].nan_to_num(7.0), dead[1].nan_to_num(7.0))
    for k in want:
        some = [0, 2] if k in ("f", "dinit") else slice(None)
        assert torch.isfinite(want[k][some]).all(), k
        assert torch.equal(got[k][some], want[k][some]), k
    init[1], dead[1] = 0, 0
    init[2] = float("inf")
    got = call(init, dead)
    for k in ("y", "dx", "ddt", "dz", "dB", "dC"):
        assert not got[k][2, c.lens[2]:].any(), k
        assert torch.equal(got[k][:2], want[k][:2]), k
