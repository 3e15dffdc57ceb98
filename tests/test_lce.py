"""Cross entropy over a large vocabulary against fp64, its gradients against
differences, masks that leave rows or everything out, and the refusals.

Tolerances: loss and lse, max|got - ref| / max(1, max|ref|) <= 1e-5 for both
storage types (bf16 products are exact in fp32 and the sums are fp32: D = 4096
terms of |x||w| about 2 / sqrt(D) each, 4096 * 6e-8 worst case times a logit's
term 0.03 = 7e-6).  Gradients ||got - ref|| / ||ref||: fp32 1e-5; bf16 4e-3 (the
result's rounding, 2^-9 / sqrt(3) = 1.1e-3, the same once more for g, and room
for values just above a power of two), and what no fp32 logit can give: a logit
l is off by about 2^-24 max|l| a few times over, which makes exp(l - lse) off by
as much of itself, and where p is near 1 that is much of p - 1: 2^-21 max|l| of
||p dloss|| ||w|| (||x|| for dw) on top.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import linear_recurrence_scan_chunked_gb300 as lrs

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
GTOL = {"f32": 1e-5, "bf16": 4e-3}


def make(N, V, D, dtype, seed=0, pad=0.1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=g).to(DT[dtype])
    w = (2 / math.sqrt(D) * torch.randn(V, D, generator=g)).to(DT[dtype])
    t = torch.randint(0, V, (N,), generator=g)
    t[torch.rand(N, generator=g) < pad] = -100
    return x, w, t, torch.randn(N, generator=g) / N


def ref(x, w, t, dloss, ignore=-100, lse_in=None):
    """lse_in: the backward pass's input, as it is given (fp32: 2^-24 of its
    size, which the exponentials of a row all share)."""
    x, w = x.double(), w.double()
    l = x @ w.T
    lse = torch.logsumexp(l, 1)
    live = (t != ignore) & (t >= 0) & (t < w.shape[0])
    at = torch.where(live, t, 0)
    loss = torch.where(live, lse - l[torch.arange(len(t)), at], 0.0)
    g = torch.softmax(l, 1) if lse_in is None else torch.exp(l - lse_in.double().cpu()[:, None])
    g[torch.arange(len(t)), at] -= 1
    g *= torch.where(live, dloss.double(), 0.0)[:, None]
    return loss, lse, g @ w, g.T @ x


def slack(x, w, t, dloss, rdx, rdw):
    """2^-21 max|l| ||p dloss|| ||w|| relative to ||dx||, and for dw."""
    x, w = x.double(), w.double()
    l = x @ w.T
    p = torch.softmax(l, 1) * torch.where(t != -100, dloss.double(), 0.0)[:, None]
    e = 2.0 ** -21 * float(l.abs().max())
    return (e * float((p.abs() @ w.abs()).norm()) / max(float(rdx.norm()), 1e-300),
            e * float((p.abs().T @ x.abs()).norm()) / max(float(rdw.norm()), 1e-300))


def dist(got, want):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all()
    n = float(want.norm())
    return float((got - want).norm()) / n if n else float(got.norm())


def mx(got, want):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape and torch.isfinite(got).all()
    return float((got - want).abs().max() / max(1.0, float(want.abs().max())))


# one of everything, exact tiles, one past and one short of them, odd widths (no 16-byte rows)
SHAPES = [(1, 1, 1), (1, 2, 8), (2, 3, 5), (1, 1000, 64), (5, 257, 64), (128, 256, 64), (129, 255, 72), (64, 128, 128),
          (200, 1000, 250), (300, 513, 33), (256, 512, 256), (257, 777, 264), (130, 5000, 1000), (1, 20000, 136),
          (1000, 130, 64), (513, 129, 1024), (40, 300, 4096), (31, 9000, 1023), (9, 140, 514),
          (33, 300, 1030), (20, 90, 516), (7, 65, 511), (6, 40, 2562)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,D", SHAPES)
def test_loss_and_gradients(cuda, N, V, D, dtype):
    x, w, t, dl = make(N, V, D, dtype, seed=N + V + D)
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
    loss, lse = cuda.lce_fwd(xd, wd, td)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    _, _, rdx, rdw = ref(x, w, t, dl, lse_in=lse)
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
    assert dx.dtype == dw.dtype == DT[dtype]
    if V > 1:  # one word: the gradient is 0 but for roundings
        sx, sw = slack(x, w, t, dl, rdx, rdw)
        assert dist(dx, rdx) <= GTOL[dtype] + sx and dist(dw, rdw) <= GTOL[dtype] + sw
    else:
        assert float(dx.abs().max()) <= 1e-6 and float(dw.abs().max()) <= 1e-6
    # the same bits again, into buffers that hold something else
    loss2, lse2 = cuda.lce_fwd(xd, wd, td, loss=torch.full_like(loss, 9.0), lse=torch.full_like(lse, 9.0))
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dx2, dw2 = cuda.lce_bwd(xd, wd, td, lse, dd, dx=torch.full_like(dx, 9.0), dw=torch.full_like(dw, 9.0))
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_than_one_piece(cuda, dtype):
    """A vocabulary of several pieces, ragged at the end, and a last tile of one word."""
    N, V, D = 70, 40001, 96
    x, w, t, dl = make(N, V, D, dtype, seed=3)
    t[0], t[1], t[2] = 0, V - 1, V - 2
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
    loss, lse = cuda.lce_fwd(xd, wd, td)
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    assert dist(dx, rdx) <= GTOL[dtype] and dist(dw, rdw) <= GTOL[dtype]


@pytest.mark.gpu
def test_many_rows(cuda):
    N, V, D = 20000, 300, 64
    x, w, t, dl = make(N, V, D, "bf16", seed=4)
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
    loss, lse = cuda.lce_fwd(xd, wd, td)
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    assert dist(dx, rdx) <= GTOL["bf16"] and dist(dw, rdw) <= GTOL["bf16"]


@pytest.mark.gpu
def test_uniform_upstream_is_not_biased(cuda):
    """dloss = 1/N, which bf16 cannot hold: the rounding of g must not shift dw as a whole."""
    N, V, D = 1021, 500, 64
    x, w, t, _ = make(N, V, D, "bf16", seed=5, pad=0.0)
    x = x.abs()  # rows that add up
    dl = torch.full((N,), 1.0 / N)
    _, _, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
    _, lse = cuda.lce_fwd(xd, wd, td)
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
    assert dist(dx, rdx) <= GTOL["bf16"] and dist(dw, rdw) <= GTOL["bf16"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_all_rows_ignored_and_other_ignore(cuda, dtype):
    x, w, t, dl = make(9, 100, 64, dtype, seed=6)
    xd, wd, dd = x.cuda(), w.cuda(), dl.cuda()
    off = torch.full((9,), -100).cuda()
    loss, lse = cuda.lce_fwd(xd, wd, off)
    assert not loss.any() and mx(lse, ref(x, w, t, dl)[1]) <= 1e-5
    dd[3] = float("inf")  # masked: must not reach the result
    dd[4] = float("nan")
    dx, dw = cuda.lce_bwd(xd, wd, off, lse, dd)
    assert not dx.any() and not dw.any()
    # a word of the vocabulary as the ignored one
    t[:] = 7
    t[2] = 8
    rl, _, rdx, rdw = ref(x, w, t, dl, ignore=7)
    dd = dl.cuda()
    loss, lse = cuda.lce_fwd(xd, wd, t.cuda(), ignore=7)
    dx, dw = cuda.lce_bwd(xd, wd, t.cuda(), lse, dd, ignore=7)
    assert mx(loss, rl) <= 1e-5 and dist(dx, rdx) <= GTOL[dtype] and dist(dw, rdw) <= GTOL[dtype]


@pytest.mark.gpu
def test_large_logits(cuda):
    """Logits of +-1e4 (sums of exponentials relative to the maximum), and a vocabulary word at -inf's edge."""
    N, V, D = 20, 700, 64
    x, w, t, dl = make(N, V, D, "f32", seed=7, pad=0.0)
    x = x * 3e3
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
    loss, lse = cuda.lce_fwd(xd, wd, td)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    # a logit near 1e4 is good to 1e4 * 1e-6: g to a few 1e-2 where the softmax is not saturated
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
    assert dist(dx, rdx) <= 5e-2 and dist(dw, rdw) <= 5e-2


@pytest.mark.gpu
def test_nan_stays_in_its_rows(cuda):
    N, V, D = 140, 300, 64
    x, w, t, dl = make(N, V, D, "bf16", seed=8, pad=0.0)
    x[5, 3] = float("nan")
    loss, lse = cuda.lce_fwd(x.cuda(), w.cuda(), t.cuda())
    bad = torch.isnan(loss).cpu()
    assert bad[5] and int(bad.sum()) == 1
    dx, _ = cuda.lce_bwd(x.cuda(), w.cuda(), t.cuda(), lse, dl.cuda())
    bad = torch.isnan(dx).any(1).cpu()
    assert bad[5] and int(bad.sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 37])
def test_ignored_rows_do_not_count_whatever_they_hold(cuda, dtype, D):
    """Rows whose target is ignored: values whose logits overflow to infinities and
    NaN leave dx = 0 there and nothing in dw (0 times a finite row); a NaN leaves
    dx = 0 as well."""
    N, V = 150, 300
    x, w, t, dl = make(N, V, D, dtype, seed=12, pad=0.0)
    t[[3, 60, 140]] = -100
    x[3] = 3e38
    x[60] = -3e38
    x[60, ::2] = 3e38
    x[140] = -3e38
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    _, _, rdx, rdw = ref(torch.where((t == -100)[:, None], torch.zeros_like(x), x), w, t, dl)
    loss, lse = cuda.lce_fwd(xd, wd, td, ignore=-100)
    assert not loss[[3, 60, 140]].any()
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dl.cuda(), ignore=-100)
    tol = 1e-5 if dtype == "f32" else 2e-2
    assert not dx[[3, 60, 140]].any()
    assert dist(dx, rdx) <= tol and dist(dw, rdw) <= tol
    x[60, 1] = float("nan")
    loss, lse = cuda.lce_fwd(x.cuda(), wd, td, ignore=-100)
    dx, _ = cuda.lce_bwd(x.cuda(), wd, td, lse, dl.cuda(), ignore=-100)
    assert not loss[60] and not dx[60].any() and dist(dx, rdx) <= tol


@pytest.mark.gpu
def test_targets_out_of_range_are_recorded(cuda):
    x, w, t, dl = make(6, 50, 64, "f32", seed=9, pad=0.0)
    t[1], t[4] = 50, -7
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    loss, lse = cuda.lce_fwd(xd, wd, td)
    assert cuda.last_error() == cuda.LR_ERR_INDEX and cuda.last_error() == cuda.LR_OK
    assert mx(loss, rl) <= 1e-5 and not loss[1] and not loss[4]
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dl.cuda())
    assert dist(dx, rdx) <= 1e-5 and dist(dw, rdw) <= 1e-5
    cuda.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned_views_batched_shapes_streams_and_empty(cuda, dtype):
    N, V, D = 12, 90, 64
    x, w, t, dl = make(N, V, D, dtype, seed=10)
    rl, _, rdx, rdw = ref(x, w, t, dl)
    bx = torch.zeros(N * D + 1, dtype=DT[dtype], device="cuda")
    bw = torch.zeros(V * D + 3, dtype=DT[dtype], device="cuda")
    xv, wv = bx[1:].view(3, 4, D), bw[3:].view(V, D)
    xv.copy_(x.view(3, 4, D))
    wv.copy_(w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    td, dd = t.view(3, 4).cuda(), dl.view(3, 4).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        loss, lse = cuda.lce_fwd(xv, wv, td)
        dx, dw = cuda.lce_bwd(xv, wv, td, lse, dd)
    s.synchronize()
    assert loss.shape == (3, 4) and mx(loss.view(-1), rl) <= 1e-5
    assert dx.shape == (3, 4, D) and dist(dx.view(N, D), rdx) <= GTOL[dtype] and dist(dw, rdw) <= GTOL[dtype]
    e = torch.empty(0, D, dtype=DT[dtype], device="cuda")
    te = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = cuda.lce_fwd(e, wv, te)
    dx, dw = cuda.lce_bwd(e, wv, te, lse, loss)
    assert loss.shape == (0,) and dx.shape == (0, D) and not dw.any()


@pytest.mark.gpu
def test_captured_into_a_graph(cuda):
    x, w, t, dl = (v.cuda() for v in make(50, 400, 128, "bf16", seed=11))
    loss, lse = cuda.lce_fwd(x, w, t)
    dx, dw = cuda.lce_bwd(x, w, t, lse, dl)
    want = [v.clone() for v in (loss, dx, dw)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cuda.lce_fwd(x, w, t, loss=loss, lse=lse)
        cuda.lce_bwd(x, w, t, lse, dl, dx=dx, dw=dw)
    for v in (loss, dx, dw):
        v.zero_()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip((loss, dx, dw), want):
        assert torch.equal(a, b)


def test_reference_gradients_against_differences():
    x, w, t, dl = make(3, 6, 4, "f32", seed=12, pad=0.0)
    x, w, t[1] = x.double(), w.double(), -100
    _, _, rdx, rdw = ref(x, w, t, dl)
    loss = lambda a, b: float((ref(a, b, t, dl)[0] * dl.double()).sum())
    for which, r in ((0, rdx), (1, rdw)):
        for at in np.ndindex(*r.shape):
            args = [[x.clone(), w.clone()] for _ in range(2)]
            args[0][which][at] += 1e-5
            args[1][which][at] -= 1e-5
            assert abs((loss(*args[0]) - loss(*args[1])) / 2e-5 - float(r[at])) <= 1e-8


def test_refusals():
    x, w, t = torch.zeros(3, 4), torch.zeros(5, 4), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        lrs.lce_fwd(x, w, t)
    with pytest.raises(ValueError):
        lrs.lce_bwd(x, w, t, x[:, 0], x[:, 0])
    lib = lrs.load()
    P = None
    f = lambda n, v, d, p=P, dt=0: lib.lce_fwd(p, p, p, -100, p, p, n, v, d, dt, P)
    b = lambda n, v, d, p=P, dt=0: lib.lce_bwd(p, p, p, -100, p, p, p, p, n, v, d, dt, P)
    for call in (f, b):
        assert call(3, 5, 4) == lrs.LR_ERR_INVALID_ARG
        assert call(3, 5, 4, dt=3) == lrs.LR_ERR_INVALID_ARG
        assert call(-1, 5, 4) == lrs.LR_ERR_INVALID_ARG
        assert call(3, 0, 4) == lrs.LR_ERR_INVALID_ARG
        assert call(3, 5, 0) == lrs.LR_ERR_INVALID_ARG
        assert call(3, 5, 65537) == lrs.LR_ERR_TOO_LARGE
        assert call(1 << 31, 5, 4) == lrs.LR_ERR_TOO_LARGE
        assert call(3, 5, 4, ctypes.c_void_p(4097)) == lrs.LR_ERR_ALIGN
    assert f(0, 5, 4) == lrs.LR_OK
    assert b(0, 5, 4) == lrs.LR_ERR_INVALID_ARG  # dw is written even for no row


@pytest.mark.gpu
def test_refusals_on_device_tensors(cuda):
    x, w, t, dl = (v.cuda() for v in make(6, 50, 64, "f32"))
    for call in (lambda: cuda.lce_fwd(x, w.bfloat16(), t), lambda: cuda.lce_fwd(x, w[:, :32], t),
                 lambda: cuda.lce_fwd(x, w, t.int()), lambda: cuda.lce_fwd(x, w, t[:3]),
                 lambda: cuda.lce_fwd(x.t(), w, t), lambda: cuda.lce_bwd(x, w, t, dl.double(), dl),
                 lambda: cuda.lce_bwd(x, w, t, dl, dl, dx=x.bfloat16())):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [1024, 4096, 16384])
def test_confident_rows_at_long_widths(cuda, D):
    """bf16, the target's p about 0.999 and its logit a sum of thousands of terms of one
    sign, which the tensor cores shrink: loss and gradients of the two passes together
    against fp64.  p - 1 takes the difference of the backward pass's logit and the
    forward pass's lse, so both have to be off by the same."""
    N, V = 32, 300
    g = torch.Generator().manual_seed(17)
    w = torch.randn(V, D, generator=g).to(torch.bfloat16)  # words nearly orthogonal
    t = torch.arange(N) % V
    x = (12.6 * w[t].float() / w[t].float().square().sum(1, keepdim=True)).to(torch.bfloat16)
    dl = torch.ones(N) / N
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    loss, lse = cuda.lce_fwd(xd, wd, td)
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dl.cuda())
    sx, sw = slack(x, w, t, dl, rdx, rdw)
    assert dist(dx, rdx) <= GTOL["bf16"] + sx and dist(dw, rdw) <= GTOL["bf16"] + sw


@pytest.mark.gpu
def test_long_sums_do_not_shrink(cuda):
    """bf16 gradients over a k loop of 131072 terms of one sign: the mean relative
    error over the 5 million results, whose roundings average out (2^-9 / sqrt(3) /
    sqrt(5e6) = 5e-7; g's roundings are independent as well), stays below 1e-5."""
    N, V, D = 4864, 131072, 1024
    g = torch.Generator(device="cuda").manual_seed(18)
    x = (0.02 * torch.randn(N, D, device="cuda", generator=g)).bfloat16()
    w = torch.rand(V, D, device="cuda", generator=g).bfloat16()
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    w[0] = 0
    dl = torch.full((N,), 1.0 / N, device="cuda")
    _, lse = cuda.lce_fwd(x, w, t)
    dx, _ = cuda.lce_bwd(x, w, t, lse, dl)
    off = n = 0.0
    wd = w.double()
    for r in range(0, N, 608):
        p = torch.exp(x[r:r + 608].double() @ wd.T - lse[r:r + 608].double()[:, None])
        want = (p @ wd) / N  # the target's word is 0
        off += float((dx[r:r + 608].double() - want).sum())
        n += float(want.sum())
    print("bias", off / n)
    assert abs(off / n) <= 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 37])
def test_words_masked_by_the_lowest_value(cuda, dtype, D):
    """Words that a bias column holds out with the type's lowest value, whole tiles of
    columns and ragged ones: their exponentials are 0, whichever comes first."""
    N, V = 70, 700
    x, w, t, dl = make(N, V, D, dtype, seed=13, pad=0.0)
    off = torch.zeros(V, dtype=torch.bool)
    off[:150] = off[300:333] = off[650:] = True
    x[:, 0] = 1.0
    w[off] = 0.0
    w[off, 0] = torch.finfo(DT[dtype]).min
    t = torch.arange(N) % 130 + 160
    rl, rz, rdx, rdw = ref(x, w, t, dl)
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    loss, lse = cuda.lce_fwd(xd, wd, td)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    dx, dw = cuda.lce_bwd(xd, wd, td, lse, dl.cuda())
    _, _, rdx, rdw = ref(x, w, t, dl, lse_in=lse)
    sx, sw = slack(x, w[~off], t, dl, rdx, rdw[~off])
    assert dist(dx, rdx) <= GTOL[dtype] + sx and dist(dw, rdw) <= GTOL[dtype] + sw
    assert not dw.cpu()[off].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_logits_of_any_finite_size(cuda, dtype):
    """Rows whose logits are of the order of 1e6 to 1e37: loss and lse to 1e-5 of the
    row's largest, where exp(l) has left every range long ago; and a row that is
    masked throughout by one very low value: V equal words."""
    N, V, D = 33, 300, 64
    x, w, t, dl = make(N, V, D, dtype, seed=14, pad=0.0)
    x = x.float() * torch.logspace(0, 37, N)[:, None]
    x[32] = 0.0
    x[32, 0] = 1.0
    w[:, 0] = 0.0
    x, w = x.to(DT[dtype]), w.clone()
    rl, rz, _, _ = ref(x, w, t, dl)
    big = (x.double() @ w.double().T).abs().amax(1).clamp(min=1.0)
    loss, lse = cuda.lce_fwd(x.cuda(), w.cuda(), t.cuda())
    assert float(((loss.double().cpu() - rl).abs() / big).max()) <= 1e-5
    assert float(((lse.double().cpu() - rz).abs() / big).max()) <= 1e-5
    dx, dw = cuda.lce_bwd(x.cuda(), w.cuda(), t.cuda(), lse, dl.cuda())
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    low = torch.zeros(V, D, dtype=DT[dtype])
    low[:, 0] = -3e38
    loss, lse = cuda.lce_fwd(x[32:].cuda(), low.cuda(), t[32:].cuda())
    assert float(lse) == float(low[0, 0]) and float(loss) == 0.0  # log V is below lse's last bit


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_an_infinite_logit_shows_in_the_gradient(cuda, dtype):
    """exp(l - lse) of an infinite lse is not 0 for every word: the row's gradient is
    NaN, like the formula's, whether the target's logit is infinite or not."""
    N, V, D = 40, 300, 64
    x, w, t, dl = make(N, V, D, dtype, seed=15, pad=0.0)
    t[7], t[8] = 200, 201
    w[200, 0], w[201, 0] = 1.0, -1.0
    x[7:9, 0] = float("inf")
    xd, wd, td = x.cuda(), w.cuda(), t.cuda()
    loss, lse = cuda.lce_fwd(xd, wd, td)
    assert not torch.isfinite(lse[7:9]).any() and not torch.isfinite(loss[7:9]).any()
    keep = (torch.arange(N) != 7) & (torch.arange(N) != 8)
    assert mx(lse.cpu()[keep], ref(x, w, t, dl)[1][keep]) <= 1e-5
    dx, _ = cuda.lce_bwd(xd, wd, td, lse, dl.cuda())
    assert torch.isnan(dx[7:9]).all() and torch.isfinite(dx.cpu()[keep]).all()


@pytest.mark.gpu
def test_infinitely_masked_words_bf16(cuda):
    """Words at -inf: loss and lse are those of the others."""
    N, V, D = 40, 300, 64
    x, w, t, dl = make(N, V, D, "bf16", seed=16, pad=0.0)
    x[:, 0] = 1.0
    off = torch.zeros(V, dtype=torch.bool)
    off[:64] = off[280:] = True
    w[off] = 0.0
    w[off, 0] = -float("inf")
    t = torch.arange(N) % 200 + 70
    rl, rz, _, _ = ref(x, w, t, dl)
    loss, lse = cuda.lce_fwd(x.cuda(), w.cuda(), t.cuda())
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5


# budget of the scratch, N, D, words past two whole pieces
PIECES = [(1 << 20, 70, 96, 1), (1 << 20, 70, 33, 700), (1 << 20, 1, 64, 5), (8 << 20, 2560, 2048, 300),
          (1 << 18, 129, 250, 255)]


def pieced(budget, N, D, more, dtype):
    """(V, plan) of a problem of two whole pieces and a last one of `more` words."""
    lrs.test_lce_budget(budget)
    V = 2 * lrs.lce_plan_info(True, dtype, True, N, 1 << 30, D)["piece"] + more
    return V, lrs.lce_plan_info(True, dtype, True, N, V, D)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("budget,N,D,more", PIECES)
def test_pieces_of_the_vocabulary(cuda, budget, N, D, more, dtype):
    """The gradients in three pieces, the last one ragged or a single word, with dx
    summed over them, and targets in each."""
    try:
        V, _ = pieced(budget, N, D, more, dtype)
        if V * D > 1 << 26:  # a few rows make long pieces
            V = (1 << 26) // D
        x, w, t, dl = make(N, V, D, dtype, seed=19)
        t[0], t[N // 2], t[N - 1] = V - 1, 0, V - 1
        xd, wd, td, dd = (v.cuda() for v in (x, w, t, dl))
        loss, lse = cuda.lce_fwd(xd, wd, td)
        dx, dw = cuda.lce_bwd(xd, wd, td, lse, dd)
        again = cuda.lce_bwd(xd, wd, td, lse, dd, dx=torch.full_like(dx, 9.0), dw=torch.full_like(dw, 9.0))
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    finally:
        lrs.test_lce_budget(0)
    xg, wg, tg, dg = xd.double(), wd.double(), td, dd.double()  # the fp64 form on the GPU: the largest is 5e10 products
    l = xg @ wg.T
    live = tg != -100
    at = torch.where(live, tg, 0)[:, None]
    rl = torch.where(live, torch.logsumexp(l, 1) - l.gather(1, at)[:, 0], 0.0)
    g = torch.exp(l - lse.double()[:, None]).scatter_add(1, at, -torch.ones_like(l[:, :1]))
    g *= torch.where(live, dg, 0.0)[:, None]
    rdx, rdw = (g @ wg).cpu(), (g.T @ xg).cpu()
    assert mx(loss, rl.cpu()) <= 1e-5
    e = 2.0 ** -21 * float(l.abs().max())
    p = torch.softmax(l, 1) * torch.where(live, dg, 0.0)[:, None]
    sx = e * float((p.abs() @ wg.abs()).norm()) / float(rdx.norm())
    sw = e * float((p.abs().T @ xg.abs()).norm()) / float(rdw.norm())
    assert dist(dx, rdx) <= GTOL[dtype] + sx and dist(dw, rdw) <= GTOL[dtype] + sw


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rounds_of_rows(cuda, dtype):
    N, V, D = 1300, 2000, 72
    x, w, t, dl = make(N, V, D, dtype, seed=20)
    rl, rz, _, _ = ref(x, w, t, dl)
    want = cuda.lce_fwd(x.cuda(), w.cuda(), t.cuda())
    try:
        lrs.test_lce_budget(1 << 16)
        assert lrs.lce_plan_info(False, dtype, True, N, V, D)["rows"] == 512
        loss, lse = cuda.lce_fwd(x.cuda(), w.cuda(), t.cuda())
    finally:
        lrs.test_lce_budget(0)
    assert mx(loss, rl) <= 1e-5 and mx(lse, rz) <= 1e-5
    assert mx(loss, want[0].cpu()) <= 1e-6


def test_plans_and_scratch():
    """The shapes above take several pieces, with and without parts of dx; the scratch
    of large problems is what the header states, whatever the number of pieces."""
    try:
        seen = set()
        for budget, N, D, more in PIECES:
            for dtype in ("f32", "bf16"):
                V, plan = pieced(budget, N, D, more, dtype)
                assert V == 2 * plan["piece"] + more
                seen.add(plan["dx_splits"] > 1)
        assert seen == {False, True}
    finally:
        lrs.test_lce_budget(0)
    for dtype, es, planes in (("bf16", 2, 1), ("f32", 4, 3)):
        for N, V, D in ((8192, 65536, 1024), (32768, 131072, 4096), (131072, 131072, 4096), (65536, 131072, 4096),
                        (1 << 20, 50000, 1024), (1, 1 << 24, 64), (4096, 1 << 20, 4096)):
            p = lrs.lce_plan_info(True, dtype, True, N, V, D)
            g = max(2 << 30, 256 * N * 2 * planes)
            packed = 6 * (N + V) * D if dtype == "f32" else 0
            several = p["piece"] < V
            parts = 4 * N * D * (p["dx_splits"] if several or p["dx_splits"] > 1 else 0)
            acc = 4 * N * D if several and dtype == "bf16" else 0
            assert p["bytes"] <= g + packed + parts + acc + (256 << 20), (dtype, N, V, D, p)
            assert p["dx_splits"] <= 2 or N * D <= 1 << 24
            f = lrs.lce_plan_info(False, dtype, True, N, V, D)
            assert f["bytes"] <= packed + (2 << 30) + (64 << 20)
    with pytest.raises(ValueError):
        lrs.lce_plan_info(True, "f16", True, 1, 1, 1)
    with pytest.raises(ValueError):
        lrs.lce_plan_info(True, "f32", True, 0, 1, 1)
    assert lrs.test_lce_budget(-1) == lrs.LR_ERR_INVALID_ARG


@pytest.mark.gpu
def test_outgrown_scratch_is_given_back(cuda):
    """Batches that grow slowly, in a process of their own: what the library holds on
    the device is its current scratch, not the sum of all that it outgrew; what a graph
    has captured stays, and the graph's replay is right after the scratch has moved."""
    import os
    import subprocess
    import sys
    code = r"""
import torch, linear_recurrence_scan_chunked_gb300 as lrs
V, D, N = 20000, 64, 6000
w, x = torch.randn(V, D, device="cuda"), torch.randn(N, D, device="cuda")
t, dl = torch.zeros(N, dtype=torch.int64, device="cuda"), torch.ones(N, device="cuda")
dx, dw, loss, lse = torch.empty_like(x), torch.empty_like(w), torch.empty_like(dl), torch.empty_like(dl)
def call(n, x=x, dx=dx):
    lrs.lce_fwd(x[:n], w, t[:n], loss=loss[:n], lse=lse[:n])
    lrs.lce_bwd(x[:n], w, t[:n], lse[:n], dl[:n], dx=dx[:n], dw=dw)
call(8)  # the kernels are loaded
torch.cuda.synchronize()
free, held = torch.cuda.mem_get_info()[0], lrs.workspace_bytes()
for n in (1000, 1500, 2000, 2600, 3400, 4500):
    call(n)
torch.cuda.synchronize()
used, grown = free - torch.cuda.mem_get_info()[0], lrs.workspace_bytes() - held
need = 1.25 * lrs.lce_plan_info(True, "f32", True, 4500, V, D)["bytes"]
assert 200 << 20 < need, need
assert grown <= need, (grown, need)
assert used <= need + (64 << 20), (used, need)
g = torch.cuda.CUDAGraph()
gx, gdx = x[:100].clone(), torch.empty_like(x[:100])
torch.cuda.synchronize()
with torch.cuda.graph(g):
    call(100, gx, gdx)
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
call(6000)  # outgrows what the graph uses
torch.cuda.synchronize()
assert before - torch.cuda.mem_get_info()[0] >= lrs.lce_plan_info(True, "f32", True, 6000, V, D)["bytes"]
call(100, gx, gdx)
torch.cuda.synchronize()
want, want_w = gdx.clone(), dw.clone()
gdx.zero_(), dw.zero_()
g.replay()
torch.cuda.synchronize()
assert torch.equal(gdx, want) and torch.equal(dw, want_w)
assert lrs.last_error() == lrs.LR_OK
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(lrs.__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,D,dtype", [(82, 23040, 79, "f32"), (82, 5000, 64, "bf16"), (300, 300, 300, "f32")])
def test_calls_one_behind_the_other(cuda, N, V, D, dtype):
    """Thousands of small calls without a wait between them, each kernel set up while
    the one before ends: the pairs of CTAs take and give back their tensor memory in
    step.  The last call's bits are the first one's."""
    import time
    x, w, t, dl = (v.cuda() for v in make(N, V, D, dtype, seed=21))
    loss, lse = cuda.lce_fwd(x, w, t)
    dx, dw = cuda.lce_bwd(x, w, t, lse, dl)
    want = [v.clone() for v in (loss, lse, dx, dw)]
    for _ in range(4):
        for _ in range(2500):
            cuda.lce_fwd(x, w, t, loss=loss, lse=lse)
            cuda.lce_bwd(x, w, t, lse, dl, dx=dx, dw=dw)
        done = torch.cuda.Event()
        done.record()
        limit = time.monotonic() + 60
        while not done.query():
            assert time.monotonic() < limit, "the calls do not end"
            time.sleep(1e-3)
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx, dw), want))
    assert cuda.last_error() == cuda.LR_OK
