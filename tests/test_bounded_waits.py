"""Waits that run out: the tiled kernels of the recurrence and of the cross entropy
with none of their copies issued (lr_test_stall) give up after a millisecond, record
LR_ERR_TIMEOUT, leave NaN in what they computed and run again afterwards.  Nothing
faults or hangs.
"""
import pytest
import torch

import linear_recurrence_scan_chunked_gb300 as lrs

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
LIMIT = 1_000_000  # ns


@pytest.fixture
def stalled(cuda):
    def run(call):
        """call() while nothing is loaded: its outputs, which the error word belongs to."""
        assert cuda.test_stall(LIMIT) == cuda.LR_OK
        try:
            out = call()
            torch.cuda.synchronize()
        finally:
            cuda.test_stall(0)
        assert cuda.last_error() == cuda.LR_ERR_TIMEOUT
        assert cuda.last_error() == cuda.LR_OK
        return out
    yield run
    cuda.test_stall(0)
    cuda.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("T,B,D", [(33, 2, 128), (300, 2, 128), (20, 40, 1024)])
def test_gated_recurrence(cuda, stalled, T, B, D, resets, dtype):
    g = torch.Generator().manual_seed(0)
    x, zr, zi, dh = (torch.randn(T, B, D, generator=g).to(DT[dtype]).cuda() for _ in range(4))
    lam, br, bi = torch.rand(D, generator=g).cuda(), torch.zeros(D).cuda(), torch.zeros(D).cuda()
    reset = (torch.rand(T, B, generator=g) < 0.2).cuda() if resets else None
    assert lrs.plan_info("glr_fwd", dtype, True, T, B * D)["tma"]
    fwd = lambda: cuda.glr_fwd(x, zr, zi, lam, br, bi, reset=reset)
    want = fwd()
    bwd = lambda: cuda.glr_bwd(x, zr, zi, lam, br, bi, want[0], dh, reset=reset)
    grads = bwd()
    for t in stalled(fwd):
        assert torch.isnan(t).all()
    out = stalled(bwd)
    assert all(torch.isnan(out[k]).all() for k in ("dx", "dzi", "dbi"))
    if not resets:  # a reset's own dzr, and what it passes on, are 0 whatever reaches it
        assert all(torch.isnan(out[k]).all() for k in ("dzr", "dlam", "dbr", "dh0"))
    assert all(torch.equal(a, b) for a, b in zip(fwd(), want))
    again = bwd()
    assert all(torch.equal(again[k], grads[k]) for k in grads)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,D", [(40, 300, 64), (300, 20000, 2056), (700, 5000, 72)])
def test_cross_entropy(cuda, stalled, N, V, D, dtype):
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(*s, generator=g).to(DT[dtype]).cuda() / 8 for s in ((N, D), (V, D)))
    t, dl = torch.randint(0, V, (N,), generator=g).cuda(), torch.ones(N).cuda()
    loss, lse = cuda.lce_fwd(x, w, t)
    want = cuda.lce_bwd(x, w, t, lse, dl)
    for out in stalled(lambda: cuda.lce_fwd(x, w, t)):
        assert torch.isnan(out).all()
    for out in stalled(lambda: cuda.lce_bwd(x, w, t, lse, dl)):
        assert torch.isnan(out).all()
    again = cuda.lce_fwd(x, w, t)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    assert all(torch.equal(a, b) for a, b in zip(cuda.lce_bwd(x, w, t, lse, dl), want))


def test_limit_is_bounded():
    assert lrs.test_stall(2_000_000_000) == lrs.LR_ERR_INVALID_ARG
    assert lrs.test_stall(0) == lrs.LR_OK
