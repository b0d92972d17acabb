"""Norm and rotation of B and C: refusals (no GPU), and the forward and the
gradients against the fp64 definition.

Bounds.  The mean of N <= 256 squares is off by at most (8 + 5 + 2) roundings
relative to itself (eight terms a lane, five joins), its reciprocal root by half
of that and two more; u = v r w by three more: 16 roundings of |u|.  The cosine
and sine are off by 2^-24 pi / 4 (the rest of a turn, at most an eighth, in fp32)
and two roundings; a turned element is a sum of two products: 24 roundings of
|u_i| + |u_j| cover all."""
import ctypes
import threading
from fractions import Fraction

import pytest
import torch

import layer_ref as R
from ssd_chunked_scan_02_b200 import build as ssd_build
from ssd_chunked_scan_02_b200 import ssd

EPS = 1e-5


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


P = 0x1000
ST = ssd.ssd_stride_t(256, 64)


@pytest.mark.parametrize("dims,want", [
    ((-1, 4, 1, 64, 64), 1), ((1, -4, 1, 64, 64), 1), ((1, 4, 0, 64, 64), 1), ((1, 4, 1, 0, 0), 1),
    ((1, 4, 1, 257, 64), 2), ((1, 4, 1, 64, 3), 1), ((1, 4, 1, 64, 66), 1), ((1, 4, 1, 64, -2), 1),
    ((1 << 31, 4, 1, 64, 64), 2), ((1, 4, 65536, 64, 64), 2)])
def test_sizes_refused(lib, dims, want):
    d = ssd.ssd_rotate_dims_t(*dims)
    n = ctypes.c_size_t(7)
    assert lib.ssd_bc_norm_rotate_fwd(P, ST, P, ST, P, P, 0, P, P, EPS, 0, P, P, d, 1, None) == want
    assert lib.ssd_bc_norm_rotate_bwd_workspace_size(d, 1, n) == want and n.value == 7


def test_pointers_refused(lib):
    d = ssd.ssd_rotate_dims_t(1, 4, 1, 64, 64)
    good = [P, ST, P, ST, P, P, 0, P, P, EPS, 0, P, P, d, 1, None]
    for i, bad in [(0, None), (0, P + 1), (1, None), (2, None), (3, None), (4, None), (4, P + 4),
                   (5, None), (7, None), (8, None), (9, -1.0), (9, float("nan")), (11, None),
                   (12, P + 8), (13, None), (14, 5)]:
        a = list(good)
        a[i] = bad
        assert lib.ssd_bc_norm_rotate_fwd(*a) == 1, i
    empty = ssd.ssd_rotate_dims_t(0, 4, 1, 64, 64)
    assert lib.ssd_bc_norm_rotate_fwd(None, ST, None, ST, None, None, 0, None, None, EPS, 0, None,
                                      None, empty, 1, None) == 0
    n = ctypes.c_size_t(0)
    assert lib.ssd_bc_norm_rotate_bwd_workspace_size(d, 1, n) == 0 and n.value > 0
    bwd = [*good[:11], P, P, 0, P, P, P, P, d, 1, P, n.value, None]
    for i, bad in [(11, None), (14, None), (16, None), (17, P + 2), (20, None), (21, n.value - 1)]:
        a = list(bwd)
        a[i] = bad
        assert lib.ssd_bc_norm_rotate_bwd(*a) == 1, i


def test_binding_refuses(lib):
    B = torch.zeros(2, 3, 2, 8)
    w, pos, fr = torch.ones(8), torch.zeros(2, 3, dtype=torch.int64), torch.ones(4)
    for bad in (dict(B=B[0]), dict(C=B[:, :2]), dict(C=B.double()), dict(B_weight=torch.ones(7)),
                dict(C_weight=torch.ones(2, 8)), dict(positions=pos.int()),
                dict(positions=pos[:, :1].expand(2, 3)), dict(freq=fr.double()),
                dict(B=B.transpose(2, 3)), dict(B=B.transpose(2, 3).contiguous().transpose(2, 3)),
                dict(B_out=B.bfloat16()), dict()):
        a = dict(B=B, C=B, B_weight=w, C_weight=w, positions=pos, freq=fr)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            ssd.ssd_bc_norm_rotate_fwd(**a)


# ------------------------------------------------------------------ on the GPU
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
CASES = [  # b, L, G, N, R, dtype, interleaved, weights per group, view, positions
    (2, 5, 1, 128, 128, "bf16", False, False, 0, "near"),
    (2, 70, 8, 128, 64, "bf16", False, True, 64, "near"),
    (3, 33, 5, 64, 64, "bf16", True, True, 8, "far"),
    (1, 1, 1, 16, 16, "bf16", False, False, 0, "far"),
    (2, 17, 3, 24, 8, "bf16", True, False, 3, "near"),      # an odd slice: element by element
    (2, 9, 2, 33, 30, "bf16", False, True, 0, "near"),      # odd rows, 15 turned pairs
    (1, 6, 2, 7, 0, "f32", False, False, 0, "near"),        # the norm alone
    (2, 40, 1, 256, 256, "f32", False, True, 4, "far"),
    (300, 1, 1, 128, 128, "bf16", False, False, 0, "far"),  # single tokens
    (2, 700, 2, 64, 48, "f32", True, True, 0, "near"),
    (1, 20, 40, 32, 32, "bf16", False, False, 0, "near"),   # more rows than a block walks at once
    (1, 3, 2, 1, 0, "f32", False, True, 0, "near"),
]


def make(case, seed=0):
    b, L, G, N, Rr, dt, inter, per, view, where = case
    g = torch.Generator().manual_seed(seed + L)
    n = lambda *s: torch.randn(s, generator=g)                          # noqa: E731
    row = G * N
    wide = n(b, L, view + 2 * row).to(DT[dt]).cuda()[..., view:]
    pos = torch.arange(L)[None, :] + torch.zeros(b, 1, dtype=torch.int64)
    if where == "far":      # far along, at and past 2^31, and before the start
        pos = pos + torch.tensor([(1 << 20) + 7, (1 << 31) - 2, -5])[torch.arange(b) % 3][:, None]
    wshape = (G, N) if per else (N,)
    return dict(B=wide[..., :row].unflatten(2, (G, N)), C=wide[..., row:].unflatten(2, (G, N)),
                wB=(1 + 0.3 * n(*wshape)).cuda(), wC=(1 + 0.3 * n(*wshape)).cuda(),
                pos=pos.cuda(), gen=g,
                freq=(10000.0 ** (-torch.arange(0, Rr, 2, dtype=torch.float32) / max(Rr, 1))).cuda())


def args(d):
    return [d[k] for k in ("B", "C", "wB", "wC", "pos", "freq")]


def turned_size(u, Rr, inter):
    """|u_i| + |u_j| for turned elements, |u_i| for the others."""
    a = u.abs().clone()
    p = torch.arange(Rr // 2)
    i, j = (2 * p, 2 * p + 1) if inter else (p, p + Rr // 2)
    s = a[..., i] + a[..., j]
    a[..., i], a[..., j] = s, s
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])) + c[5])
def test_forward(lib, case):
    inter = case[6]
    d = make(case)
    out = ssd.ssd_bc_norm_rotate_fwd(*args(d), eps=EPS, interleaved=inter)
    zero = torch.zeros_like(d["pos"]).cpu()
    for k, got in zip("BC", out):
        a = (R.f64(d[k]), R.f64(d["w" + k]))
        ref = R.norm_rotate(*a, d["pos"].cpu(), d["freq"].cpu(), EPS, inter)
        u = R.norm_rotate(*a, zero, d["freq"].cpu(), EPS, inter)
        R.within(k, got, ref, 24 * R.U * turned_size(u, case[4], inter))


@pytest.mark.gpu
@pytest.mark.parametrize("gt", ["same", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:5])) + c[5])
def test_gradients(lib, case, gt):
    """dv = r (d - v r^2 mean(d v)), d = du w: with M = mean |d v| r^2 |v| + |d|, off by
    at most 24 roundings (the turn) + 16 (the mean and r) + 16 (r) of r M, 64 in
    all.  dweight sums du v r over the tokens: those of one block in turn (tokens /
    592 blocks, at least a tile's 32), at most 128 slots, then 592 blocks in
    eight columns."""
    b, L, G, N, Rr, dt, inter, per, view, where = case
    d = make(case, 50)
    T = DT[dt] if gt == "same" else torch.float32
    gB, gC = (torch.randn(b, L, G, N, generator=d["gen"]).to(T).cuda() for _ in range(2))
    g = ssd.ssd_bc_norm_rotate_bwd(*args(d), gB, gC, eps=EPS, interleaved=inter)
    for k, up in (("B", gB), ("C", gC)):
        v, w = R.f64(d[k]).requires_grad_(), R.f64(d["w" + k]).requires_grad_()
        out = R.norm_rotate(v, w, d["pos"].cpu(), d["freq"].cpu(), EPS, inter)
        rv, rw = torch.autograd.grad((out * R.f64(up)).sum(), (v, w))
        v, w = v.detach(), w.detach()
        r = 1 / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)
        size = turned_size(R.f64(up), Rr, inter)              # bounds |du|
        dd = size * w.abs()
        M = (dd * v.abs()).mean(-1, keepdim=True) * r * r * v.abs() + dd
        R.within("d" + k, g["d" + k], rv, 64 * R.U * r * M)
        sums = (size * v.abs() * r).sum((0, 1) if per else (0, 1, 2))
        steps = 48 + max(32, b * L / 592) + 128 + 592 * G / 8 + 8
        R.within("dw" + k, g["dw" + k], rw, steps * R.U * sums)


@pytest.mark.gpu
def test_gradients_against_differences(lib):
    """Central differences of the fp64 definition; see the convolution's test."""
    case = (2, 9, 3, 32, 16, "f32", False, True, 0, "near")
    d = make(case, 9)
    gB, gC = (torch.randn(2, 9, 3, 32, generator=d["gen"]).cuda() for _ in range(2))
    g = ssd.ssd_bc_norm_rotate_bwd(*args(d), gB, gC, eps=EPS)
    for k, up in (("B", gB), ("C", gC)):
        for key, which in (("d" + k, k), ("dw" + k, "w" + k)):
            base = {k: R.f64(d[k]), "w" + k: R.f64(d["w" + k])}
            v = torch.randn(base[which].shape, generator=d["gen"], dtype=torch.float64)

            def loss(h):
                a = {**base, which: base[which] + h * v}
                return (R.norm_rotate(a[k], a["w" + k], d["pos"].cpu(), d["freq"].cpu(), EPS, False)
                        * R.f64(up)).sum()
            want = float(loss(1e-5) - loss(-1e-5)) / 2e-5
            got = R.f64(g[key]) * v
            assert abs(float(got.sum()) - want) <= 1e-5 * float(got.abs().sum()), key


@pytest.mark.gpu
def test_rows_of_zeros_and_infinities(lib):
    """A row of zeros stays zero and its gradient finite; an infinity or a NaN
    spoils its own row and no other."""
    d = make((1, 4, 1, 64, 64, "bf16", False, False, 0, "near"))
    B, C = d["B"].clone(), d["C"].clone()
    B[0, 0], B[0, 1, 0, 3], B[0, 2, 0, 5] = 0, float("inf"), float("nan")
    up = torch.randn(1, 4, 1, 64, generator=d["gen"]).cuda()
    a = (B, C, *args(d)[2:])
    ob, oc = ssd.ssd_bc_norm_rotate_fwd(*a, eps=EPS)
    g = ssd.ssd_bc_norm_rotate_bwd(*a, up, up, eps=EPS)
    assert not ob[0, 0].any() and torch.isfinite(g["dB"][0, 0].float()).all()
    assert torch.isfinite(ob[0, 3].float()).all() and torch.isfinite(oc.float()).all()
    assert torch.isnan(ob[0, 2].float()).all() and torch.isfinite(g["dB"][0, 3].float()).all()


@pytest.mark.gpu
def test_streams_graphs_repeats_and_no_tokens(lib):
    d = make((2, 300, 4, 128, 128, "bf16", True, True, 8, "near"), 3)
    up = torch.randn(2, 300, 4, 128, generator=d["gen"]).cuda()
    flat = lambda r: [*r[0], *r[1].values()]                                    # noqa: E731
    call = lambda **k: (ssd.ssd_bc_norm_rotate_fwd(*args(d), interleaved=True, **k),   # noqa: E731
                        ssd.ssd_bc_norm_rotate_bwd(*args(d), up, up, interleaved=True, **k))
    one = flat(call())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    two = flat(call(stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = flat(call())
    d["B"].mul_(-3)
    d["pos"].add_(11)
    graph.replay()
    want = flat(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and not torch.equal(one[0], kept[0])
    e = make((2, 0, 4, 64, 64, "bf16", False, True, 0, "near"))
    B, C = ssd.ssd_bc_norm_rotate_fwd(*args(e))
    g = ssd.ssd_bc_norm_rotate_bwd(*args(e), B, C)
    assert B.shape == (2, 0, 4, 64) and not g["dwB"].any() and not g["dwC"].any()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [
    (1, 1, 1, 128, 128, "bf16", False, False, 0, "near"),   # one token: eight places, one taken
    (2, 5, 1, 128, 64, "bf16", True, False, 0, "near"),
    (8, 2048, 1, 128, 128, "bf16", False, False, 0, "near"),  # tiles of 28 tokens in eight places
    (3, 33, 5, 64, 64, "f32", True, True, 8, "near"),
    (2, 9, 2, 33, 30, "bf16", False, True, 0, "near"),      # element by element
    (1, 40, 16, 128, 0, "bf16", False, True, 0, "near"),    # every place taken
], ids=lambda c: "x".join(map(str, c[:5])) + c[5])
def test_no_epsilon(lib, case):
    """eps = 0 is the plain norm.  Places of a tile that hold no token (the last
    tokens of a tile, a single token of one group) have no norm and must not
    reach the weights' gradients.  Bounds: test_forward's and test_gradients'."""
    b, L, G, N, Rr, dt, inter, per, view, where = case
    d = make(case, 70)
    gB, gC = (torch.randn(b, L, G, N, generator=d["gen"]).cuda() for _ in range(2))
    out = ssd.ssd_bc_norm_rotate_fwd(*args(d), eps=0.0, interleaved=inter)
    g = ssd.ssd_bc_norm_rotate_bwd(*args(d), gB, gC, eps=0.0, interleaved=inter)
    for k, up, got in (("B", gB, out[0]), ("C", gC, out[1])):
        v, w = R.f64(d[k]).requires_grad_(), R.f64(d["w" + k]).requires_grad_()
        ref = R.norm_rotate(v, w, d["pos"].cpu(), d["freq"].cpu(), 0.0, inter)
        rv, rw = torch.autograd.grad((ref * R.f64(up)).sum(), (v, w))
        v, w = v.detach(), w.detach()
        r = 1 / torch.sqrt(v.square().mean(-1, keepdim=True))
        R.within(k, got, ref, 24 * R.U * turned_size(v * r * w, Rr, inter))
        size = turned_size(R.f64(up), Rr, inter)
        dd = size * w.abs()
        M = (dd * v.abs()).mean(-1, keepdim=True) * r * r * v.abs() + dd
        R.within("d" + k, g["d" + k], rv, 64 * R.U * r * M)
        sums = (size * v.abs() * r).sum((0, 1) if per else (0, 1, 2))
        steps = 48 + max(32, b * L / 592) + 128 + 592 * G / 8 + 8
        R.within("dw" + k, g["dw" + k], rw, steps * R.U * sums)


@pytest.mark.gpu
def test_calls_from_two_threads(lib):
    """Two host threads, a stream each, gradients that need different amounts of
    shared memory (128 and 64 turned elements): neither's calls fail, and both give
    what they give alone."""
    made = []
    for Rr in (128, 64):
        d = make((8, 2048, 1, 128, Rr, "bf16", False, False, 0, "near"), 90 + Rr)
        up = torch.randn(8, 2048, 1, 128, generator=d["gen"]).cuda()
        alone = ssd.ssd_bc_norm_rotate_bwd(*args(d), up, up)
        dims, n = ssd.ssd_rotate_dims_t(8, 2048, 1, 128, Rr), ctypes.c_size_t(0)
        assert lib.ssd_bc_norm_rotate_bwd_workspace_size(dims, ssd.SSD_BF16, n) == 0
        out = {k: torch.empty_like(v) for k, v in alone.items()}
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        row = [ssd.ssd_stride_t(*d[k].stride()[:2]) for k in "BC"]
        p = {k: d[k].data_ptr() for k in ("B", "C", "wB", "wC", "pos", "freq")}
        call = [p["B"], row[0], p["C"], row[1], p["wB"], p["wC"], 0, p["pos"], p["freq"], 1e-5, 0,
                up.data_ptr(), up.data_ptr(), 1, *(v.data_ptr() for v in out.values()), dims,
                ssd.SSD_BF16, ws.data_ptr(), n.value]
        made.append((call, torch.cuda.Stream(), alone, out, (d, up, ws)))
    torch.cuda.synchronize()
    start, status = threading.Barrier(2), [set(), set()]

    def work(i):
        call, stream = made[i][:2]
        start.wait()
        for _ in range(4000):
            status[i].add(lib.ssd_bc_norm_rotate_bwd(*call, stream.cuda_stream))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{ssd.SSD_OK}, {ssd.SSD_OK}]
    for _, _, alone, out, _ in made:
        assert all(torch.equal(alone[k], out[k]) for k in alone)


@pytest.mark.gpu
@pytest.mark.parametrize("case", [(2, 9, 2, 64, 32, "f32", False, True, 0, "near"),
                                  (1, 5, 3, 33, 20, "bf16", True, True, 0, "far")],
                         ids=lambda c: "x".join(map(str, c[:5])) + c[5])
def test_frequencies_that_are_no_numbers(lib, case):
    """An infinite or NaN frequency gives NaN where its pair goes (also at position
    0: 0 * inf) and in that pair's weights' gradients; the other pairs are what
    they are without it."""
    b, L, G, N, Rr, inter = *case[:5], case[6]
    d = make(case, 80)
    up = torch.randn(b, L, G, N, generator=d["gen"]).cuda()
    a = args(d)
    bad = [1, 4, Rr // 2 - 1]
    a[5] = d["freq"].clone()
    a[5][bad] = torch.tensor([float("nan"), float("inf"), -float("inf")]).cuda()
    spoilt = torch.zeros(N, dtype=torch.bool, device="cuda")
    for p in bad:
        spoilt[[2 * p, 2 * p + 1] if inter else [p, p + Rr // 2]] = True
    want = ssd.ssd_bc_norm_rotate_fwd(*args(d), interleaved=inter)
    got = ssd.ssd_bc_norm_rotate_fwd(*a, interleaved=inter)
    gw = ssd.ssd_bc_norm_rotate_bwd(*args(d), up, up, interleaved=inter)
    gg = ssd.ssd_bc_norm_rotate_bwd(*a, up, up, interleaved=inter)
    for o, w in [*zip(got, want), (gg["dwB"], gw["dwB"]), (gg["dwC"], gw["dwC"])]:
        assert torch.isnan(o[..., spoilt]).all()
        assert torch.equal(o[..., ~spoilt], w[..., ~spoilt])


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.mark.gpu
def test_far_positions(lib):
    """Positions up to 2^40, against angles in exact arithmetic.  Beside
    test_forward's bound, a step is 2^-64 of a turn off at most."""
    b, L, G, N, Rr = 6, 2, 1, 64, 64
    d = make((b, L, G, N, Rr, "f32", False, False, 0, "near"), 60)
    base = torch.tensor([(1 << 31) - 1, (1 << 32) + 5, (1 << 36) + 12345, (1 << 40) - 77, -(1 << 38) - 3,
                         (1 << 33) + 1])
    pos = base[:, None] + torch.arange(L)
    freq = torch.cat((torch.tensor([1.0, 0.99999994, 3.0, 100.25]),
                      10000.0 ** (-torch.arange(4, 32, dtype=torch.float32) / 32)))
    turns = [[[Fraction(int(p)) * Fraction(float(f)) / (2 * PI) for f in freq] for p in row] for row in pos]
    ang = torch.tensor([[[float((t - round(t)) * 2 * PI) for t in r] for r in row] for row in turns],
                       dtype=torch.float64)
    out = ssd.ssd_bc_norm_rotate_fwd(d["B"], d["C"], d["wB"], d["wC"], pos.cuda(), freq.cuda(), eps=EPS)
    c, s = ang.cos()[:, :, None], ang.sin()[:, :, None]
    for k, got in zip("BC", out):
        v = R.f64(d[k])
        u = v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS) * R.f64(d["w" + k])
        p, q = u[..., :32], u[..., 32:]
        ref = torch.cat((p * c - q * s, p * s + q * c), -1)
        step = 2 * float(PI) * 2.0 ** -64 * pos.abs().double()[:, :, None, None]
        R.within(k, got, ref, (24 * R.U + step) * turned_size(u, Rr, False))
