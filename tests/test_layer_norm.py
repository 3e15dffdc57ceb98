"""Layer norm forward and backward against fp64, its gradient against
differences, and the refusals.

Tolerances on max|got - ref| / max(1, max|ref|): fp32 2e-6 for the rows (sums of
D <= 16384 terms in trees of depth about 20: 20 * 6e-8 = 1.2e-6), bf16 storage
2^-8 (one rounding of values below 2 max: 2^-9 of max|ref|, and the norm of a
rounded sum); the column sums over N rows relative to the sum of their terms'
magnitudes, 2e-6 (chains of at most a few hundred terms, then a tree).
"""
import ctypes

import numpy as np
import pytest
import torch

import linear_recurrence_scan_chunked_gb300 as lrs

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 2e-6, "bf16": 2.0 ** -8}


def make(N, D, dtype, seed=0, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    return dict(x=(1.5 * rn(N, D) + shift).to(DT[dtype]), res=rn(N, D).to(DT[dtype]), dy=rn(N, D).to(DT[dtype]),
                dres=rn(N, D).to(DT[dtype]), w=1 + 0.2 * rn(D), b=0.2 * rn(D))


def ref_fwd(x, w, b, eps):
    x = x.double()
    mean = x.mean(-1)
    rstd = 1 / ((x - mean[..., None]).square().mean(-1) + eps).sqrt()
    return (x - mean[..., None]) * rstd[..., None] * w.double() + (0 if b is None else b.double()), mean, rstd


def ref_bwd(x, w, mean, rstd, dy, dres):
    xh = (x.double() - mean.double()[..., None]) * rstd.double()[..., None]
    t = dy.double() * w.double()
    dx = (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True)) * rstd.double()[..., None]
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy.double() * xh), dy.double()


def err(got, ref):
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    return float((got - ref).abs().max() / max(1.0, float(ref.abs().max()))) if ref.numel() else 0.0


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 8), (9, 33), (1, 1024), (8, 1024), (1000, 64), (333, 257), (70, 1111),
          (64, 2048), (33, 2052), (40, 4096), (17, 4099), (9, 6000), (5, 8192), (3, 8193), (3, 12000), (2, 16384),
          (4000, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", SHAPES)
def test_fwd_bwd(cuda, N, D, dtype):
    c = make(N, D, dtype, seed=N + D)
    d = {k: v.cuda() for k, v in c.items()}
    # plain, and with the residual: the sum is rounded to the storage type, the norm is of the rounded sum
    y, mean, rstd = cuda.layer_norm_fwd(d["x"], d["w"], d["b"])
    ry, rm, rr = ref_fwd(c["x"], c["w"], c["b"], 1e-5)
    for got, ref, tol in ((y, ry, TOL[dtype]), (mean, rm, 2e-6)):
        assert err(got, ref) <= tol
    assert float(((rstd.double().cpu() - rr) / rr).abs().max()) <= 4e-6
    y, mean, rstd, s = cuda.layer_norm_fwd(d["x"], d["w"], d["b"], res=d["res"], eps=1e-3)
    want = (c["x"].float() + c["res"].float()).to(DT[dtype])
    assert torch.equal(s.cpu(), want)
    ry, rm, rr = ref_fwd(want, c["w"], c["b"], 1e-3)
    assert err(y, ry) <= TOL[dtype] and err(mean, rm) <= 2e-6
    # backward, with and without the residual stream's gradient
    for dres in (None, "dres"):
        got = cuda.layer_norm_bwd(s, d["w"], mean, rstd, d["dy"], dres=d[dres] if dres else None)
        dx, tw, tb = ref_bwd(want, c["w"], mean.cpu(), rstd.cpu(), c["dy"], c[dres] if dres else None)
        assert err(got["dx"], dx) <= 2 * TOL[dtype]
        for k, t in (("dw", tw), ("db", tb)):
            e = (got[k].double().cpu() - t.sum(0)).abs() / t.abs().sum(0).clamp(min=1.0)
            assert float(e.max()) <= 2e-6, k
    again = cuda.layer_norm_bwd(s, d["w"], mean, rstd, d["dy"], dres=d["dres"],
                                out={k: torch.full_like(v, 3.0) for k, v in got.items()})
    for k in got:
        assert torch.equal(again[k], got[k]), k


@pytest.mark.gpu
def test_many_rows(cuda):
    """More rows than CTAs by far, and a number that leaves the last round short."""
    c = make(20011, 96, "bf16", seed=3)
    d = {k: v.cuda() for k, v in c.items()}
    y, mean, rstd = cuda.layer_norm_fwd(d["x"], d["w"])
    assert err(y, ref_fwd(c["x"], c["w"], None, 1e-5)[0]) <= TOL["bf16"]
    got = cuda.layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"])
    dx, tw, tb = ref_bwd(c["x"], c["w"], mean.cpu(), rstd.cpu(), c["dy"], None)
    assert err(got["dx"], dx) <= 2 * TOL["bf16"]
    for k, t in (("dw", tw), ("db", tb)):
        assert float(((got[k].double().cpu() - t.sum(0)).abs() / t.abs().sum(0)).max()) <= 2e-6


@pytest.mark.gpu
def test_large_mean_does_not_cancel(cuda):
    """Rows whose mean is a thousand times their spread: the variance is taken of the deviations."""
    x = (1000.0 + torch.randn(6, 640, generator=torch.Generator().manual_seed(1)))
    _, _, rstd = cuda.layer_norm_fwd(x.cuda(), torch.ones(640).cuda())
    rr = ref_fwd(x, torch.ones(640), None, 1e-5)[2]
    # the mean is good to 1000 * 1e-7 of a spread of 1: the variance to its square
    assert float(((rstd.double().cpu() - rr) / rr).abs().max()) <= 1e-5


@pytest.mark.gpu
def test_constant_rows_and_infinities(cuda):
    x = torch.full((4, 130), 3.25, device="cuda")
    w, b = torch.ones(130, device="cuda"), torch.full((130,), 0.5, device="cuda")
    y, mean, rstd = cuda.layer_norm_fwd(x, w, b)
    assert torch.equal(y, torch.full_like(y, 0.5)) and torch.equal(mean, x[:, 0])
    x[1, 7] = float("inf")
    x[2, 0] = float("nan")
    y, _, _ = cuda.layer_norm_fwd(x, w, b)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[3]).all()
    assert torch.isnan(y[1]).any() and torch.isnan(y[2]).all()


@pytest.mark.gpu
def test_unaligned_views_streams_and_empty(cuda):
    c = make(37, 64, "bf16", seed=4)
    buf = torch.zeros(37 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    x = buf[1:].view(37, 64)  # contiguous, 2-byte aligned only
    x.copy_(c["x"])
    w = c["w"].cuda()
    want, mean, rstd = cuda.layer_norm_fwd(c["x"].cuda(), w)
    y, _, _ = cuda.layer_norm_fwd(x, w)
    assert err(y, ref_fwd(c["x"], c["w"], None, 1e-5)[0]) <= TOL["bf16"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    cuda.layer_norm_fwd(c["x"].cuda(), w, y=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    e = torch.empty(0, 64, device="cuda")
    y, mean, rstd = cuda.layer_norm_fwd(e, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    got = cuda.layer_norm_bwd(e, w, mean, rstd, e)
    assert not got["dw"].any() and not got["db"].any()


def test_reference_gradient_against_differences():
    c = {k: v.double() for k, v in make(3, 5, "f32", seed=6).items()}
    _, mean, rstd = ref_fwd(c["x"], c["w"], c["b"], 1e-5)
    dx, tw, tb = ref_bwd(c["x"], c["w"], mean, rstd, c["dy"], None)
    ref = dict(x=dx, w=tw.sum(0), b=tb.sum(0))
    loss = lambda e: float((ref_fwd(e["x"], e["w"], e["b"], 1e-5)[0] * c["dy"]).sum())
    for name in ("x", "w", "b"):
        for at in np.ndindex(*c[name].shape):
            up, dn = ({**c, name: c[name].clone()} for _ in range(2))
            up[name][at] += 1e-5
            dn[name][at] -= 1e-5
            assert abs((loss(up) - loss(dn)) / 2e-5 - float(ref[name][at])) <= 1e-7, (name, at)


def test_refusals():
    x, w = torch.zeros(3, 4), torch.zeros(4)
    with pytest.raises(ValueError):
        lrs.layer_norm_fwd(x, w)
    with pytest.raises(ValueError):
        lrs.layer_norm_bwd(x, w, x[:, 0], x[:, 0], x)
    lib = lrs.load()
    P, f = None, ctypes.c_float
    assert lib.layer_norm_fwd(*([P] * 8), 3, 4, f(1e-5), 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.layer_norm_fwd(*([P] * 8), 3, 4, f(-1.0), 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.layer_norm_fwd(*([P] * 8), 3, 4, f(float("nan")), 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.layer_norm_fwd(*([P] * 8), 3, 0, f(1e-5), 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.layer_norm_fwd(*([P] * 8), 3, 16385, f(1e-5), 0, P) == lrs.LR_ERR_TOO_LARGE
    assert lib.layer_norm_fwd(*([P] * 8), 0, 4, f(1e-5), 0, P) == lrs.LR_OK
    assert lib.layer_norm_bwd(*([P] * 9), 3, 4, 9, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.layer_norm_bwd(*([P] * 9), 3, 4, 0, P) == lrs.LR_ERR_INVALID_ARG
    odd = ctypes.c_void_p(ctypes.addressof(ctypes.create_string_buffer(64)) + 1)
    assert lib.layer_norm_fwd(odd, P, odd, P, odd, P, odd, odd, 1, 1, f(1e-5), 0, P) == lrs.LR_ERR_ALIGN


@pytest.mark.gpu
def test_refusals_on_device_tensors(cuda):
    d = {k: v.cuda() for k, v in make(4, 8, "f32").items()}
    for call in (lambda: cuda.layer_norm_fwd(d["x"].t(), d["w"]), lambda: cuda.layer_norm_fwd(d["x"], d["w"][:4]),
                 lambda: cuda.layer_norm_fwd(d["x"], d["w"].double()),
                 lambda: cuda.layer_norm_fwd(d["x"], d["w"], res=d["res"].bfloat16()),
                 lambda: cuda.layer_norm_fwd(d["x"], d["w"], s=d["res"]),
                 lambda: cuda.layer_norm_bwd(d["x"], d["w"], d["x"][:, 0], d["w"], d["dy"])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 9, 24, 31, 32, 49, 63, 64, 65, 100, 104, 119, 128, 250, 255, 257, 511, 520, 900, 1500, 1792, 2047, 3000, 5000, 10995, 16383])
def test_every_instance(cuda, D, dtype):
    """The row shapes between the sizes above: each number of elements a thread, the wide rows."""
    c = make(67, D, dtype, seed=D)
    d = {k: v.cuda() for k, v in c.items()}
    y, mean, rstd = cuda.layer_norm_fwd(d["x"], d["w"], d["b"])
    ry, rm, _ = ref_fwd(c["x"], c["w"], c["b"], 1e-5)
    assert err(y, ry) <= TOL[dtype] and err(mean, rm) <= 2e-6
    got = cuda.layer_norm_bwd(d["x"], d["w"], mean, rstd, d["dy"], dres=d["dres"])
    dx, tw, tb = ref_bwd(c["x"], c["w"], mean.cpu(), rstd.cpu(), c["dy"], c["dres"])
    assert err(got["dx"], dx) <= 2 * TOL[dtype]
    for k, t in (("dw", tw), ("db", tb)):
        assert float(((got[k].double().cpu() - t.sum(0)).abs() / t.abs().sum(0).clamp(min=1.0)).max()) <= 2e-6, k


@pytest.mark.gpu
def test_outputs_belong_to_the_stream_that_writes_them(cuda):
    """Memory that the caching allocator has just taken back on the current stream may
    still be read there: an output written on another stream is not made of it."""
    x = torch.randn(8192, 1, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    t = torch.zeros(8192, 1, dtype=torch.int64, device="cuda")
    rows = torch.randn(8192, 128, device="cuda")
    pool = torch.zeros(8192, 128, device="cuda")
    lse = torch.ones(8192, 1, device="cuda")
    s = torch.cuda.Stream()

    def step(**k):
        pool.zero_()
        torch.cuda.synchronize()
        return cuda.glr_step(rows, rows, rows, w, w, w, pool, **k)

    for call in (lambda **k: cuda.layer_norm_fwd(x, w, **k)[0], lambda **k: cuda.layer_norm_bwd(x, w, lse, lse, x, **k)["dx"],
                 lambda **k: cuda.glr_fwd(x, x, x, w, w, w, **k)[0], lambda **k: cuda.glr_bwd(x, x, x, w, w, w, x, x, **k)["dx"],
                 step,
                 lambda **k: cuda.lce_bwd(x, rows, t, lse, lse, **k)[0], lambda **k: cuda.lr_scan_fwd(x, x, **k),
                 lambda **k: cuda.sru_fwd(x, x, x, x, w, w, **k)[0]):
        want = call()
        torch.cuda.synchronize()
        old = torch.empty_like(x)
        taken = old.data_ptr()
        del old
        y = call(stream=s)
        assert y.data_ptr() != taken
        s.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_calls_from_several_threads(cuda):
    """The forward call takes no lock and the binding gives up the GIL: threads on
    streams of their own, each through shapes that the others ask for first as well."""
    import threading
    shapes = [(4000, 128), (900, 1111), (300, 4096), (100, 8200), (5000, 49)]
    data = [make(N, D, "f32", seed=N) for N, D in shapes]
    xs, ws = [d["x"].cuda() for d in data], [d["w"].cuda() for d in data]
    torch.cuda.synchronize()
    got = {}

    def work(k):
        s = torch.cuda.Stream()
        for i in range(20):
            j = (i * 3 + k) % len(shapes)
            got[k, i] = (j, cuda.layer_norm_fwd(xs[j], ws[j], stream=s)[0])
        s.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    want = [cuda.layer_norm_fwd(x, w)[0] for x, w in zip(xs, ws)]
    assert len(got) == 160 and all(torch.equal(y, want[j]) for j, y in got.values())
