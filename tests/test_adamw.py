"""AdamW over many tensors, moments in fp32 and in 8 bits, against fp64 and (the
codes) against the same separately rounded fp32 operations in numpy.

Tolerances: fp32 moments a few roundings of 2^-24; a weight 2^-23 |p| for its own
rounding and 1e-6 of the distance that the step moves it (the roundings of m, v,
the root, the quotient and the products, 2^-24 each), taken as at least 10 lr.
"""
import ctypes

import numpy as np
import pytest
import torch

import linear_recurrence_scan_chunked_gb300 as lrs

H = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 255, 256, 257, 4096, 4097, 0, 10000, 33, 70001]


def make(sizes, gdtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda n, s=1.0: s * torch.randn(n, generator=g)
    return dict(p=[rn(n, 0.02) for n in sizes], g=[rn(n, 1e-2).to(gdtype) for n in sizes],
                m=[rn(n, 1e-2) for n in sizes], v=[rn(n, 1e-2).square() for n in sizes])


def ref_step(p, g, m, v, step, scale=1.0):
    g = g.double() * scale
    m = H["beta1"] * m.double() + (1 - H["beta1"]) * g
    v = H["beta2"] * v.double() + (1 - H["beta2"]) * g * g
    mh, vh = m / (1 - H["beta1"] ** step), v / (1 - H["beta2"] ** step)
    return p.double() * (1 - H["lr"] * H["weight_decay"]) - H["lr"] * mh / (vh.sqrt() + H["eps"]), m, v


def check_p(got, ref, before):
    e = (got.double().cpu() - ref).abs()
    moved = (ref - before.double()).abs().clamp(min=10 * H["lr"])
    assert bool((e <= 2.0 ** -23 * ref.abs() + 1e-6 * moved).all())


@pytest.mark.gpu
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scaled", [False, True])
def test_step_32(cuda, gdtype, scaled):
    c = make(SIZES, gdtype)
    d = {k: [t.cuda() for t in v] for k, v in c.items()}
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in SIZES]
    s = torch.tensor([0.625], device="cuda") if scaled else None
    cuda.adamw_step(d["p"], d["g"], d["m"], d["v"], step=3, grad_scale=s, copies=copies, **H)
    for i in range(len(SIZES)):
        rp, rm, rv = ref_step(c["p"][i], c["g"][i], c["m"][i], c["v"][i], 3, 0.625 if scaled else 1.0)
        check_p(d["p"][i], rp, c["p"][i])
        assert torch.allclose(d["m"][i].double().cpu(), rm, rtol=0, atol=2.0 ** -22 * 0.1)
        assert torch.allclose(d["v"][i].double().cpu(), rv, rtol=2.0 ** -21, atol=0)
        assert torch.equal(copies[i], d["p"][i].bfloat16())


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_unaligned_tensors_and_more_than_one_launch(cuda, eight):
    """950 tensors, views at odd offsets of one buffer: three launches, the
    scalar path, the hash of the tensor's index in the call."""
    sizes = [1 + (i * 37) % 600 for i in range(950)]
    offs = np.concatenate([[0], np.cumsum(np.array(sizes) + 1)])
    c = make(sizes, torch.float32, seed=2)

    def view(ts, dt=torch.float32):
        buf = torch.zeros(int(offs[-1]) + 1, dtype=dt, device="cuda")
        vs = [buf[int(o) + 1:int(o) + 1 + n] for o, n in zip(offs, sizes)]
        for a, b in zip(vs, ts):
            a.copy_(b)
        return buf, vs

    pb, p = view(c["p"])
    _, g = view(c["g"])
    if eight:
        _, m = view([torch.zeros(n) for n in sizes], torch.int8)
        _, v = view([torch.zeros(n) for n in sizes], torch.uint8)
        _, _, ms, vs = cuda.adamw8_state(p)
        cuda.adamw8_step(p, g, m, v, ms, vs, step=1, seed=9, **H)
        for i in (0, 399, 400, 800, 949):
            rm, rv, _, _ = np_moments(c["g"][i].numpy(), np.zeros(sizes[i], np.float32), np.zeros(sizes[i], np.float32))
            qm, sm = np_encode_m(rm, np_noise(sizes[i], 9, i)[0])
            qv, sv = np_encode_v(rv, np_noise(sizes[i], 9, i)[1])
            assert np.array_equal(m[i].cpu().numpy(), qm) and np.array_equal(ms[i].cpu().numpy(), sm)
            assert np.array_equal(v[i].cpu().numpy(), qv) and np.array_equal(vs[i].cpu().numpy(), sv)
    else:
        _, m = view(c["m"])
        _, v = view(c["v"])
        cuda.adamw_step(p, g, m, v, step=1, **H)
    for i in range(0, 950, 13):
        z = torch.zeros(sizes[i])
        check_p(p[i], ref_step(c["p"][i], c["g"][i], z if eight else c["m"][i], z if eight else c["v"][i], 1)[0],
                c["p"][i])
    gaps = torch.ones(pb.numel(), dtype=torch.bool)
    for o, n in zip(offs, sizes):
        gaps[int(o) + 1:int(o) + 1 + n] = False
    assert not pb.cpu()[gaps].any()  # nothing written between the tensors


# ---- the 8-bit codes in numpy: every operation rounded to fp32 by itself

F = np.float32


def np_noise(n, seed, tensor):
    M = (1 << 32) - 1
    out = []
    for i in range(n):
        h = (i + tensor * 0x9E3779B1 + seed * 0xBB67AE85) & M
        h = ((h ^ (h >> 16)) * 0x6A09E667) & M
        h = ((h ^ (h >> 15)) * 0x3C6EF373) & M
        out.append(h ^ (h >> 16))
    h = np.array(out, dtype=np.int64).reshape(-1)
    return (h >> 16).astype(F) / F(65536), (h & 0xFFFF).astype(F) / F(65536)


def np_moments(g, m, v):
    c1, c2 = F(1 - H["beta1"]), F(1 - H["beta2"])
    g = g.astype(F)
    return F(H["beta1"]) * m + c1 * g, F(H["beta2"]) * v + c2 * (g * g), None, None


def np_scale(x):
    nb = -(-len(x) // 256)
    pad = np.zeros(nb * 256, F)
    pad[:len(x)] = np.abs(x)
    s = pad.reshape(nb, 256).max(1)
    inv = np.where(s > 0, F(1) / np.where(s > 0, s, F(1)), F(0)).astype(F)
    return s, (pad.reshape(nb, 256) * inv[:, None]).reshape(-1)[:len(x)]


def np_encode_m(m, u):
    s, r = np_scale(m)
    q = np.minimum(np.floor(np.sqrt(r) * F(127) + u), 127)
    return np.where(m < 0, -q, q).astype(np.int8), s


def np_encode_v(v, u):
    s, r = np_scale(v)
    q = np.minimum(np.floor(np.sqrt(np.sqrt(r)) * F(255) + u), 255)
    return np.where((v > 0) & (q < 1), 1, q).astype(np.uint8), s


def np_decode(qm, sm, qv, sv):
    n = len(qm)
    t = qm.astype(F) * F(1 / 127.0)
    m = (t * np.abs(t)) * np.repeat(sm, 256)[:n]
    t = qv.astype(F) * F(1 / 255.0)
    t = t * t
    return m, (t * t) * np.repeat(sv, 256)[:n]


@pytest.mark.gpu
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
def test_step_8_bits(cuda, gdtype):
    """Three steps: codes, scales and values equal to the numpy operations bit for bit, weights to fp64."""
    sizes = [1, 5, 256, 257, 1000, 0, 4100]
    c = make(sizes, gdtype, seed=5)
    d = {k: [t.cuda() for t in v] for k, v in c.items()}
    m, v, ms, vs = cuda.adamw8_state(d["p"])
    copies = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
    have = [np_decode(np.zeros(n, np.int8), np.zeros(-(-n // 256), F), np.zeros(n, np.uint8),
                      np.zeros(-(-n // 256), F)) for n in sizes]
    for step in (1, 2, 3):
        g = [(t.float() * (1 + step)).to(gdtype) for t in c["g"]]
        before = [t.clone() for t in d["p"]]
        cuda.adamw8_step(d["p"], [t.cuda() for t in g], m, v, ms, vs, step=step, seed=100 + step, copies=copies, **H)
        mv, vv = cuda.adamw8_values(m, v, ms, vs)
        for i, n in enumerate(sizes):
            rp, _, _ = ref_step(before[i].cpu(), g[i], torch.from_numpy(have[i][0]), torch.from_numpy(have[i][1]), step)
            check_p(d["p"][i], rp, before[i].cpu())
            nm, nv, _, _ = np_moments(g[i].float().numpy(), *have[i])
            um, uv = np_noise(n, 100 + step, i)
            qm, sm = np_encode_m(nm, um)
            qv, sv = np_encode_v(nv, uv)
            assert np.array_equal(m[i].cpu().numpy(), qm) and np.array_equal(v[i].cpu().numpy(), qv)
            assert np.array_equal(ms[i].cpu().numpy(), sm) and np.array_equal(vs[i].cpu().numpy(), sv)
            have[i] = np_decode(qm, sm, qv, sv)
            assert np.array_equal(mv[i].cpu().numpy(), have[i][0]) and np.array_equal(vv[i].cpu().numpy(), have[i][1])
            assert torch.equal(copies[i], d["p"][i].bfloat16())


def test_codes_are_right_in_the_mean():
    """The rounding of the rooted values is unbiased and never off by a code step (CPU)."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal(256).astype(F)
    acc = np.zeros(256)
    rounds = 400
    for seed in range(rounds):
        q, s = np_encode_m(x, np_noise(256, seed, 3)[0])
        root = np.sqrt(np.abs(x) / s[0]) * 127
        assert np.all(np.abs(np.abs(q.astype(float)) - root) < 1 + 1e-4)
        acc += np.abs(q) - root
    # each rounding's variance is at most 1/4: the mean of 400 within 5 sigma, and 16 bits of noise
    assert np.abs(acc / rounds).max() <= 5 * 0.5 / rounds ** 0.5 + 2.0 ** -16


@pytest.mark.gpu
def test_zero_gradients_and_nonfinite(cuda):
    p = [torch.ones(300, device="cuda")]
    m, v, ms, vs = cuda.adamw8_state(p)
    g = [torch.zeros(300, device="cuda")]
    cuda.adamw8_step(p, g, m, v, ms, vs, step=1, seed=1, **H)
    assert torch.allclose(p[0], torch.full_like(p[0], 1 - H["lr"] * H["weight_decay"]))
    assert not m[0].any() and not v[0].any() and not ms[0].any()
    # an infinite gradient stays in its own tensor (fp32 moments: in its own element)
    g32 = [torch.zeros(300, device="cuda"), torch.zeros(300, device="cuda")]
    g32[0][5] = float("inf")
    q = [torch.ones(300, device="cuda") for _ in range(2)]
    z = lambda: [torch.zeros(300, device="cuda") for _ in range(2)]
    cuda.adamw_step(q, g32, z(), z(), step=1, **H)
    assert not torch.isfinite(q[0][5]) and int(torch.isfinite(q[0]).sum()) == 299 and torch.isfinite(q[1]).all()


def test_refusals():
    t = [torch.zeros(4)]
    with pytest.raises(ValueError):
        lrs.adamw_step(t, t, t, t, step=1, lr=1e-3)
    lib = lrs.load()
    P = None
    n = (ctypes.c_int64 * 1)(4)
    ptr = (ctypes.c_void_p * 1)(4096)
    odd = (ctypes.c_void_p * 1)(4097)
    nul = (ctypes.c_void_p * 1)(None)
    f = lambda count, nn, p, step=1, b1=0.9, gd=0, eps=1e-8: lib.adamw_step(
        count, nn, p, p, p, p, P, step, 1e-3, b1, 0.95, eps, 0.1, P, gd, P)
    assert f(-1, n, ptr) == lrs.LR_ERR_INVALID_ARG
    assert f(0, P, P) == lrs.LR_OK
    assert f(1, P, P) == lrs.LR_ERR_INVALID_ARG
    assert f(1, n, nul) == lrs.LR_ERR_INVALID_ARG
    assert f(1, n, odd) == lrs.LR_ERR_ALIGN
    assert f(1, n, ptr, step=0) == lrs.LR_ERR_INVALID_ARG
    assert f(1, n, ptr, b1=1.0) == lrs.LR_ERR_INVALID_ARG
    assert f(1, n, ptr, eps=float("nan")) == lrs.LR_ERR_INVALID_ARG
    assert f(1, n, ptr, gd=2) == lrs.LR_ERR_INVALID_ARG
    assert f(1, (ctypes.c_int64 * 1)(-3), ptr) == lrs.LR_ERR_INVALID_ARG
    assert f(1, (ctypes.c_int64 * 1)(0), nul) == lrs.LR_OK  # an empty tensor needs no memory
    assert lib.adamw8_step(1, n, ptr, ptr, ptr, ptr, P, P, P, 1, 1e-3, 0.9, 0.95, 1e-8, 0.1, P, 1, 0,
                           P) == lrs.LR_ERR_INVALID_ARG


@pytest.mark.gpu
def test_refusals_on_device_tensors(cuda):
    t = [torch.zeros(8, device="cuda")]
    h = [torch.zeros(8, device="cuda", dtype=torch.float16)]
    for call in (lambda: cuda.adamw_step(t, t, t, [t[0][:4]], step=1, lr=1e-3),
                 lambda: cuda.adamw_step(t, t, t, t + t, step=1, lr=1e-3),
                 lambda: cuda.adamw_step(t, t, [t[0].double()], t, step=1, lr=1e-3),
                 lambda: cuda.adamw_step(t, t, t, t, step=1, lr=1e-3, copies=t),
                 lambda: cuda.adamw_step(t, t, t, t, step=1, lr=1e-3, grad_scale=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        cuda.adamw_step(t, h, t, t, step=1, lr=1e-3)


def test_vector_path_needs_what_its_accesses_need():
    """The element path wherever an address does not allow the widths that the kernels
    access with: 16 bytes of fp32 weights, moments and of the values of both codes, 8
    of bf16 gradients and copies, 4 of codes (CPU: fake addresses, no access)."""
    lib, base = lrs.load(), 1 << 20
    # kind, gradient type, bytes of (p, g, m, v, copy)
    for kind, gd, need in ((0, 0, (16, 16, 16, 16, 8)), (0, 1, (16, 8, 16, 16, 8)), (1, 0, (16, 16, 4, 4, 8)),
                           (1, 1, (16, 8, 4, 4, 8)), (2, 0, (16, 16, 4, 4, 16))):
        assert lib.lr_test_adamw_vec(kind, gd, *[base] * 5) == 1
        for at, bytes_ in enumerate(need):
            for off in range(1, 16):
                ptr = [base] * 5
                ptr[at] += off
                assert lib.lr_test_adamw_vec(kind, gd, *ptr) == (off % bytes_ == 0), (kind, gd, at, off)


@pytest.mark.gpu
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_values_into_views_at_any_offset(cuda, off, which):
    """fp32 outputs of the codes' values at 4, 8 and 12 bytes past a vector's start."""
    n = 1030
    g = torch.Generator().manual_seed(6)
    m = [torch.randint(-127, 128, (n,), dtype=torch.int8, generator=g).cuda()]
    v = [torch.randint(0, 256, (n,), dtype=torch.uint8, generator=g).cuda()]
    ms, vs = [torch.rand(5, generator=g).cuda()], [torch.rand(5, generator=g).cuda()]
    want = cuda.adamw8_values(m, v, ms, vs)
    buf = torch.zeros(n + 4, device="cuda")
    out = [[torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]]
    out[which] = [buf[off:off + n]]
    got = cuda.adamw8_values(m, v, ms, vs, *out)
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[1][0], want[1][0])
    assert not buf[:off].any() and not buf[off + n:].any()


def ratio(x, s):
    """x / s in blocks of 256 as the codes take it, also where 1 / s is past fp32's
    largest number: both times 2^64 then, which is exact."""
    up = F(2.0 ** 64)
    tiny = (s > 0) & (s < F(2.0 ** -120))
    inv = np.where(s > 0, F(1) / np.where(tiny, s * up, np.where(s > 0, s, F(1))), F(0)).astype(F)
    k = np.repeat(tiny, 256)[:len(x)]
    return np.where(k, np.abs(x) * up, np.abs(x)).astype(F) * np.repeat(inv, 256)[:len(x)]


def block_max(x):
    return np.array([np.abs(x[i:i + 256]).max() for i in range(0, len(x), 256)], F)


@pytest.mark.gpu
@pytest.mark.parametrize("vec", [True, False])
def test_8_bits_moments_too_small_to_invert(cuda, vec):
    """Blocks whose largest v, or m, is a positive number whose reciprocal fp32 does
    not hold, beside elements without any gradient: weights to fp64, codes and scales
    bit for bit."""
    sizes = [4 * 256 + 40, 300, 256, 256]
    g = [torch.zeros(n) for n in sizes]
    rng = np.random.default_rng(3)
    for b, mag in enumerate((1e-18, 1e-19, 1e-20, 1e-21, 3e-19)):  # v about 5e-38 .. 5e-44
        at = rng.integers(0, 40, 5) + 256 * b
        g[0][at] = torch.from_numpy(rng.standard_normal(5).astype(F)) * mag
    g[1][::7] = 1e-20
    g[2][::3] = 2e-38  # m subnormal, v = 0
    g[3][5], g[3][6] = 1e-21, 1.0
    buf = [torch.ones(n + 1, device="cuda") for n in sizes]
    p = [b[:-1] if vec else b[1:] for b in buf]
    for t in p:
        t.copy_(torch.from_numpy(rng.standard_normal(t.numel()).astype(F)))
    m, v, ms, vs = cuda.adamw8_state(p)
    have = [(np.zeros(n, F), np.zeros(n, F)) for n in sizes]
    for step in (1, 2, 3):
        before = [t.cpu().clone() for t in p]
        cuda.adamw8_step(p, [t.cuda() for t in g], m, v, ms, vs, step=step, seed=step, **H)
        for i, n in enumerate(sizes):
            rp, _, _ = ref_step(before[i], g[i], torch.from_numpy(have[i][0]), torch.from_numpy(have[i][1]), step)
            assert torch.isfinite(p[i]).all()
            check_p(p[i], rp, before[i])
            nm, nv, _, _ = np_moments(g[i].numpy(), *have[i])
            um, uv = np_noise(n, step, i)
            sm, sv = block_max(nm), block_max(nv)
            qm = np.minimum(np.floor(np.sqrt(ratio(nm, sm)) * F(127) + um), 127)
            qv = np.minimum(np.floor(np.sqrt(np.sqrt(ratio(nv, sv))) * F(255) + uv), 255)
            qm, qv = np.where(nm < 0, -qm, qm).astype(np.int8), np.where((nv > 0) & (qv < 1), 1, qv).astype(np.uint8)
            assert np.array_equal(ms[i].cpu().numpy(), sm) and np.array_equal(vs[i].cpu().numpy(), sv)
            assert np.array_equal(m[i].cpu().numpy(), qm) and np.array_equal(v[i].cpu().numpy(), qv)
            have[i] = np_decode(qm, sm, qv, sv)


@pytest.mark.gpu
@pytest.mark.parametrize("width", [64, 256])
def test_8_bits_an_embedding_whose_tokens_stay_away(cuda, width):
    """One row of an embedding gets a gradient once; 1500 steps of zero gradients
    take the block's v through the subnormal numbers.  Weights against fp64 from the
    moments that the codes stood for, every step."""
    p = [torch.randn(16, width, generator=torch.Generator().manual_seed(1)).cuda()]
    g = torch.zeros(16, width)
    g[::4] = 1e-4 * torch.randn(4, width, generator=torch.Generator().manual_seed(2))
    m, v, ms, vs = cuda.adamw8_state(p)
    zero, g = torch.zeros_like(p[0]), g.cuda()
    worst = torch.zeros((), device="cuda", dtype=torch.float64)
    for step in range(1, 1501):
        have = cuda.adamw8_values(m, v, ms, vs)
        before = p[0].clone()
        now = g if step == 1 else zero
        cuda.adamw8_step(p, [now], m, v, ms, vs, step=step, seed=step, **H)
        rp, _, _ = ref_step(before, now, have[0][0].view_as(now), have[1][0].view_as(now), step)
        bound = 2.0 ** -23 * rp.abs() + 1e-6 * (rp - before.double()).abs().clamp(min=10 * H["lr"])
        over = ((p[0].double() - rp).abs() / bound).max()
        worst = torch.maximum(worst, torch.nan_to_num(over, nan=1e9))
    assert float(worst) <= 1.0
    assert 0 < float(vs[0].max()) < 2.9e-39  # the range was reached


@pytest.mark.gpu
def test_8_bits_an_infinite_gradient_moves_no_other_weight(cuda):
    g = 1e-2 * torch.randn(256, generator=torch.Generator().manual_seed(4))
    g[5] = float("inf")
    p = [torch.ones(256, device="cuda")]
    cuda.adamw8_step(p, [g.cuda()], *cuda.adamw8_state(p), step=1, seed=1, **H)
    z = torch.zeros(256)
    rp, _, _ = ref_step(torch.ones(256), g, z, z, 1)
    keep = torch.arange(256) != 5
    assert not torch.isfinite(p[0][5])
    check_p(p[0].cpu()[keep], rp[keep], torch.ones(255))


@pytest.mark.gpu
def test_8_bits_a_v_far_below_its_block(cuda):
    """v / scale below fp32's numbers and no eps to hide it: the step is lr all the same
    (v itself is a subnormal of 3500 units, its root good to 7e-5)."""
    g = torch.full((256,), 1e-20)
    g[9] = 1e3
    p = [torch.ones(256, device="cuda")]
    cuda.adamw8_step(p, [g.cuda()], *cuda.adamw8_state(p), step=1, seed=1, lr=1e-2, beta1=0.9, beta2=0.95, eps=0.0,
                     weight_decay=0.0)
    assert torch.allclose(p[0], torch.full_like(p[0], 0.99), rtol=0, atol=1e-6 + 1e-2 * 1e-4)
