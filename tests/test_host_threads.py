"""Calls from two host threads, each on its own stream and at sizes that need
different amounts of shared memory: none fails, and each gives what it gives alone."""
import threading

import pytest
import torch

from ssd_chunked_scan_02_b200 import build as ssd_build
from ssd_chunked_scan_02_b200 import ssd


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


def inputs(P, N, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g).cuda()                       # noqa: E731
    b, L, H = 2, 128, 2
    return dict(x=n(b, L, H, P), dt=n(b, L, H).abs() * 0.1, A=-n(H).abs(), B=n(b, L, 1, N), C=n(b, L, 1, N),
                D=n(H), h=n(b, H, P, N))


def forward(d, chunk):
    need = ssd.ssd_chunk_scan_fwd_workspace_size(ssd._fwd_dims(d["x"], d["B"]), chunk, torch.float32)
    ws, y, f = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), torch.empty_like(d["x"]), \
        torch.empty_like(d["h"])
    run = lambda stream: ssd.ssd_chunk_scan_fwd(                            # noqa: E731
        *(d[k] for k in ("x", "dt", "A", "B", "C", "D")), chunk, y=y, final_states=f, workspace=ws,
        stream=stream)
    return run, (y, f)


def correction(d, _):
    """(adds to its output: each call starts from what is there, zero at first)"""
    need = ssd.ssd_state_correction_workspace_size(ssd._fwd_dims(d["x"], d["C"]), torch.float32)
    ws, y = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), torch.zeros_like(d["x"])
    run = lambda stream: ssd.ssd_state_correction_fwd(                      # noqa: E731
        d["h"], d["dt"], d["A"], d["C"], y, workspace=ws, stream=stream)
    return run, (y,)


@pytest.mark.gpu
@pytest.mark.parametrize("make", [forward, correction], ids=["forward", "correction"])
def test_fp32_calls_at_two_sizes(lib, make):
    calls = 1500
    sizes = [(128, 256, 64), (64, 32, 16)]              # head, states, chunk
    alone = []
    for i, (P, N, chunk) in enumerate(sizes):
        run, out = make(inputs(P, N, i), chunk)
        for _ in range(calls):
            run(None)
        alone.append(out)
    torch.cuda.synchronize()
    work = [(*make(inputs(P, N, i), chunk), torch.cuda.Stream()) for i, (P, N, chunk) in enumerate(sizes)]
    torch.cuda.synchronize()
    start, errors = threading.Barrier(2), []

    def loop(run, _, stream):
        start.wait()
        try:
            for _ in range(calls):
                run(stream)
        except ssd.SSDError as e:
            errors.append(str(e))
    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert errors == []
    for (_, out, _), want in zip(work, alone):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
