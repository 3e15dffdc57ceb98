"""Gated linear recurrence: the kernels against a step-by-step fp64 loop, the
loop's gradients against differences, the single-token step, and the refusals.

Tolerances, max|got - ref| / max(1, max|ref|) as in the other parity tests:
fp32 1e-5 (the decay is good to about 1e-7 and a state remembers at most a few
hundred steps of independent roundings: sqrt(500) 1e-7 = 2e-6), bf16 storage
2e-2 (a few roundings of 2^-9 each).  Sums over all steps are compared
relative to the sum of their terms' magnitudes, at the same tolerances.
"""
import ctypes

import numpy as np
import pytest
import torch

import linear_recurrence_scan_chunked_gb300 as lrs

TOL = {"f32": 1e-5, "bf16": 2e-2}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NAMES = ("x", "zr", "zi", "lam", "br", "bi")


def make(T, B, D, dtype, seed=0, resets="some", h0=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    d = {k: rn(T, B, D).to(DT[dtype]) for k in ("x", "zr", "zi", "dh")}
    d["lam"] = -8.0 * torch.log(0.9 + 0.099 * torch.rand(D, generator=g))
    d["br"], d["bi"] = 0.5 * rn(D), 0.5 * rn(D)
    d["h0"] = rn(B, D) if h0 else None
    d["dh_last"] = rn(B, D) if h0 else None
    if resets == "none":
        d["reset"] = None
    elif resets == "all":
        d["reset"] = torch.ones(T, B, dtype=torch.uint8)
    else:
        d["reset"] = (torch.rand(T, B, generator=g) < 0.05).to(torch.uint8) * 3
    return d


def ref_fwd(d):
    """The recurrence as it is written down, in fp64, one step after the other."""
    x, zr, zi, lam, br, bi = (d[k].double() for k in NAMES)
    T, B, D = x.shape
    s = d["h0"].double() if d["h0"] is not None else torch.zeros(B, D, dtype=torch.float64)
    out = torch.empty(T, B, D, dtype=torch.float64)
    for t in range(T):
        r, i = torch.sigmoid(zr[t] + br), torch.sigmoid(zi[t] + bi)
        a = torch.exp(-lam * r)
        f = torch.sqrt(-torch.expm1(-2 * lam * r))
        if d["reset"] is not None:
            k = (d["reset"][t] != 0)[:, None]
            a, f = torch.where(k, 0.0, a), torch.where(k, 1.0, f)
        s = a * s + f * i * x[t]
        out[t] = s
    return out, s


def ref_bwd(d, h):
    x, zr, zi, lam, br, bi = (d[k].double() for k in NAMES)
    T, B, D = x.shape
    z = torch.zeros(B, D, dtype=torch.float64)
    h0 = d["h0"].double() if d["h0"] is not None else z
    w = d["dh_last"].double() if d["dh_last"] is not None else z
    o = {k: torch.empty(T, B, D, dtype=torch.float64) for k in ("dx", "dzr", "dzi")}
    sums = {k: torch.zeros(D, dtype=torch.float64) for k in ("dlam", "dbr", "dbi")}
    mags = {k: torch.zeros(D, dtype=torch.float64) for k in sums}
    for t in range(T - 1, -1, -1):
        r, i = torch.sigmoid(zr[t] + br), torch.sigmoid(zi[t] + bi)
        a = torch.exp(-lam * r)
        f = torch.sqrt(-torch.expm1(-2 * lam * r))
        hp = h[t - 1].double() if t else h0
        dd = d["dh"][t].double() + w
        dloga = dd * (a * hp - i * x[t] * a * a / f)
        if d["reset"] is not None:
            k = (d["reset"][t] != 0)[:, None]
            a, f, dloga = torch.where(k, 0.0, a), torch.where(k, 1.0, f), torch.where(k, 0.0, dloga)
        o["dx"][t] = dd * f * i
        o["dzi"][t] = dd * f * x[t] * i * (1 - i)
        o["dzr"][t] = -lam * dloga * r * (1 - r)
        for k, v in (("dlam", -dloga * r), ("dbr", o["dzr"][t]), ("dbi", o["dzi"][t])):
            sums[k] += v.sum(0)
            mags[k] += v.abs().sum(0)
        w = a * dd
    return dict(o, dh0=w, **sums), mags


def dev(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def err(got, ref):
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any()
    return float((got - ref).abs().max() / max(1.0, float(ref.abs().max()))) if ref.numel() else 0.0


# every carry protocol and both paths: one step, look-back, chain, strip (wide), walker (long), odd widths
SHAPES = [(1, 1, 1), (1, 3, 128), (2, 2, 4), (33, 3, 7), (257, 2, 130), (300, 2, 128), (1021, 1, 257),
          (70, 130, 132), (96, 20, 1024), (2100, 16, 64), (9000, 1, 36), (9001, 1, 128), (5000, 2, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_fwd_bwd(cuda, shape, dtype):
    d = make(*shape, dtype, seed=sum(shape))
    c = dev(d)
    args = [c[k] for k in NAMES]
    h, last = cuda.glr_fwd(*args, h0=c["h0"], reset=c["reset"])
    rh, rlast = ref_fwd(d)
    assert h.dtype == DT[dtype] and last.dtype == torch.float32
    assert err(h, rh) <= TOL[dtype]
    assert err(last, rlast) <= 1e-5  # the state is not rounded to the storage type
    # backward from the stored h on both sides
    hs = h.cpu()
    got = cuda.glr_bwd(*args, h, c["dh"], h0=c["h0"], reset=c["reset"], dh_last=c["dh_last"])
    ref, mags = ref_bwd(d, hs)
    for k in ("dx", "dzr", "dzi"):
        assert err(got[k], ref[k]) <= TOL[dtype], k
    assert err(got["dh0"], ref["dh0"]) <= 1e-5
    for k in ("dlam", "dbr", "dbi"):
        e = ((got[k].double().cpu() - ref[k]).abs() / mags[k].clamp(min=1.0)).max()
        assert float(e) <= 1e-5, k
    # the same bits again, and into buffers that hold something else
    out = {k: torch.full_like(v, 7.0) for k, v in got.items()}
    again = cuda.glr_bwd(*args, h, c["dh"], h0=c["h0"], reset=c["reset"], dh_last=c["dh_last"], out=out)
    for k in got:
        assert torch.equal(again[k], got[k]), k


@pytest.mark.gpu
@pytest.mark.parametrize("resets", ["none", "all"])
def test_resets_none_and_all(cuda, resets):
    d = make(130, 3, 128, "f32", seed=5, resets=resets)
    c = dev(d)
    args = [c[k] for k in NAMES]
    h, last = cuda.glr_fwd(*args, h0=c["h0"], reset=c["reset"])
    rh, rlast = ref_fwd(d)
    assert err(h, rh) <= 1e-5 and err(last, rlast) <= 1e-5
    got = cuda.glr_bwd(*args, h, c["dh"], h0=c["h0"], reset=c["reset"], dh_last=c["dh_last"])
    ref, _ = ref_bwd(d, h.cpu())
    for k in ref:
        assert err(got[k], ref[k]) <= 1e-5 * (1 if got[k].dim() > 1 else 130), k
    if resets == "all":  # nothing before a step reaches it: not even an infinite initial state
        assert not got["dzr"].any() and not got["dh0"].any() and not got["dlam"].any()


@pytest.mark.gpu
def test_reset_as_bool_and_no_states(cuda):
    d = make(64, 2, 128, "f32", seed=6, h0=False)
    c = dev(d)
    args = [c[k] for k in NAMES]
    h, last = cuda.glr_fwd(*args, reset=c["reset"].bool(), want_last=False)
    assert last is None
    assert err(h, ref_fwd(d)[0]) <= 1e-5
    got = cuda.glr_bwd(*args, h, c["dh"], reset=c["reset"].bool(), want_dh0=False)
    assert got.get("dh0") is None
    assert err(got["dx"], ref_bwd(d, h.cpu())[0]["dx"]) <= 1e-5


@pytest.mark.gpu
def test_saturated_gates(cuda):
    """Gates at 0 and 1 to the last bit, a decay of exactly 1 (nothing enters, the
    gradient of the decay is 0, not NaN) and one of exactly 0."""
    T, B, D = 40, 1, 8
    d = make(T, B, D, "f32", seed=7, resets="none")
    d["zr"][:] = torch.tensor([-200.0, 200.0, -30.0, 30.0, 0.0, 5.0, -5.0, 1.0])
    d["zi"][:] = torch.tensor([200.0, -200.0, 30.0, -30.0, 0.0, 5.0, -5.0, 1.0])
    d["lam"] = torch.tensor([1.0, 500.0, 1e-3, 2.0, 0.0, 30.0, 1e-6, 0.25])
    c = dev(d)
    args = [c[k] for k in NAMES]
    h, _ = cuda.glr_fwd(*args, h0=c["h0"])
    assert err(h, ref_fwd(d)[0]) <= 1e-5
    assert torch.equal(h[-1, 0, 0].cpu(), d["h0"][0, 0]) and torch.equal(h[-1, 0, 4].cpu(), d["h0"][0, 4])
    got = cuda.glr_bwd(*args, h, c["dh"], h0=c["h0"], dh_last=c["dh_last"])
    for k in got:
        assert torch.isfinite(got[k]).all(), k
    keep = [1, 2, 3, 5, 6, 7]  # where the decay is not exactly 1
    ref, _ = ref_bwd(d, h.cpu())
    assert err(got["dx"][:, :, keep], ref["dx"][:, :, keep]) <= 1e-5
    assert not got["dzr"][:, :, [0, 4]].any()


@pytest.mark.gpu
def test_long_memory_keeps_its_input_scale(cuda):
    """lam sigma(zr) down to 1e-7: 1 - a^2 must not cancel (f = sqrt(2 lam r))."""
    d = make(50, 1, 128, "f32", seed=8, resets="none")
    d["lam"] = torch.logspace(-7, -1, 128)
    d["h0"] = torch.zeros(1, 128)
    c = dev(d)
    h, _ = cuda.glr_fwd(*[c[k] for k in NAMES], h0=c["h0"])
    rh = ref_fwd(d)[0]
    rel = (h.double().cpu() - rh).abs().amax((0, 1)) / rh.abs().amax((0, 1))
    assert float(rel.max()) <= 1e-5


@pytest.mark.gpu
def test_pieces_are_the_whole(cuda):
    """A sequence in two pieces, the fp32 state handed over and its gradient back."""
    d = make(200, 2, 128, "bf16", seed=9)
    c = dev(d)
    P = [c[k] for k in ("lam", "br", "bi")]
    cut = 77
    whole, last = cuda.glr_fwd(*[c[k] for k in NAMES], h0=c["h0"], reset=c["reset"])
    lo = [c[k][:cut] for k in ("x", "zr", "zi")]
    hi = [c[k][cut:].contiguous() for k in ("x", "zr", "zi")]
    h1, s1 = cuda.glr_fwd(*lo, *P, h0=c["h0"], reset=c["reset"][:cut])
    h2, s2 = cuda.glr_fwd(*hi, *P, h0=s1, reset=c["reset"][cut:].contiguous())
    assert err(torch.cat([h1, h2]), whole) <= 2e-2
    assert err(s2, last) <= 1e-5
    g2 = cuda.glr_bwd(*hi, *P, h2, c["dh"][cut:].contiguous(), h0=s1, reset=c["reset"][cut:].contiguous(),
                      dh_last=c["dh_last"])
    g1 = cuda.glr_bwd(*lo, *P, h1, c["dh"][:cut], h0=c["h0"], reset=c["reset"][:cut], dh_last=g2["dh0"])
    g = cuda.glr_bwd(*[c[k] for k in NAMES], whole, c["dh"], h0=c["h0"], reset=c["reset"], dh_last=c["dh_last"])
    assert err(torch.cat([g1["dzr"], g2["dzr"]]), g["dzr"]) <= 2e-2
    assert err(g1["dh0"], g["dh0"]) <= 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 1024), (7, 130), (5, 129), (300, 64), (2, 8192)])
def test_step(cuda, B, D, dtype):
    d = make(1, B, D, dtype, seed=B + D)
    c = dev(d)
    n_slots = B + 3
    g = torch.Generator().manual_seed(1)
    pool = torch.randn(n_slots, D, generator=g)
    slots = torch.randperm(n_slots, generator=g)[:B].to(torch.int32)
    if B > 2:
        slots[1] = -1
    state = pool.cuda()
    args = [c[k][0].contiguous() if c[k].dim() == 3 else c[k] for k in NAMES]
    h = cuda.glr_step(*args, state, slots=slots.cuda(), reset=c["reset"][0].contiguous())
    want, rows = pool.double().clone(), torch.zeros(B, D, dtype=torch.float64)
    for b, slot in enumerate(slots.tolist()):
        if slot >= 0:
            one = {k: (v[:, b:b + 1] if k in ("x", "zr", "zi", "reset") else v) for k, v in d.items()}
            one["h0"] = pool[slot:slot + 1]
            rows[b] = ref_fwd(one)[1][0]
            want[slot] = rows[b]
    assert err(state, want) <= 1e-6 * 4
    assert err(h, rows) <= TOL[dtype]
    untouched = [s for s in range(n_slots) if s not in slots.tolist()]
    assert torch.equal(state.cpu()[untouched], pool[untouched])
    assert cuda.last_error() == cuda.LR_OK


@pytest.mark.gpu
def test_step_follows_forward(cuda):
    """Decoding token by token gives the sequence form's fp32 state."""
    d = make(40, 3, 128, "bf16", seed=12)
    c = dev(d)
    _, last = cuda.glr_fwd(*[c[k] for k in NAMES], h0=c["h0"], reset=c["reset"])
    state = c["h0"].clone()
    for t in range(40):
        cuda.glr_step(c["x"][t], c["zr"][t], c["zi"][t], c["lam"], c["br"], c["bi"], state, reset=c["reset"][t])
    assert err(state, last) <= 1e-5


@pytest.mark.gpu
def test_step_slot_past_the_pool_is_recorded(cuda):
    d = dev(make(1, 3, 128, "f32"))
    args = [d[k][0].contiguous() if d[k].dim() == 3 else d[k] for k in NAMES]
    pool = torch.ones(2, 128, device="cuda")
    slots = torch.tensor([0, 2, -5], dtype=torch.int32, device="cuda")
    h = cuda.glr_step(*args, pool, slots=slots)
    assert cuda.last_error() == cuda.LR_ERR_INDEX
    assert cuda.last_error() == cuda.LR_OK
    assert not h[1].any() and not h[2].any() and h[0].any()
    assert torch.equal(pool[1], torch.ones(128, device="cuda"))


@pytest.mark.gpu
def test_empty_sequences(cuda):
    d = dev(make(1, 2, 8, "f32"))
    e = {k: d[k][:0] for k in ("x", "zr", "zi", "dh")}
    P = [d[k] for k in ("lam", "br", "bi")]
    h, last = cuda.glr_fwd(e["x"], e["zr"], e["zi"], *P, h0=d["h0"])
    assert h.shape == (0, 2, 8) and torch.equal(last, d["h0"])
    g = cuda.glr_bwd(e["x"], e["zr"], e["zi"], *P, h, e["dh"], h0=d["h0"], dh_last=d["dh_last"])
    assert torch.equal(g["dh0"], d["dh_last"])
    assert not g["dlam"].any() and not g["dbr"].any() and not g["dbi"].any()


@pytest.mark.gpu
def test_other_stream_and_graph(cuda):
    d = dev(make(300, 2, 128, "f32", seed=3))
    args = [d[k] for k in NAMES]
    want, _ = cuda.glr_fwd(*args, h0=d["h0"], reset=d["reset"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    h, last = torch.empty_like(want), torch.empty_like(d["h0"])
    cuda.glr_fwd(*args, h0=d["h0"], reset=d["reset"], h=h, h_last=last, stream=s)
    s.synchronize()
    assert torch.equal(h, want)
    g = torch.cuda.CUDAGraph()
    h.zero_()
    with torch.cuda.graph(g):
        cuda.glr_fwd(*args, h0=d["h0"], reset=d["reset"], h=h, h_last=last)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want)


def test_reference_gradients_against_differences():
    """The fp64 loop's gradients, as the tests above use them, against central
    differences of the forward loop (CPU): error about step^2 = 1e-10."""
    d = {k: (v.double() if v is not None and v.is_floating_point() else v)
         for k, v in make(6, 2, 3, "f32", seed=4, resets="some").items()}
    d["reset"] = torch.zeros(6, 2, dtype=torch.uint8)
    d["reset"][3, 1] = 1

    def loss(e):
        h, last = ref_fwd(e)
        return float((h * e["dh"]).sum() + (last * e["dh_last"]).sum())

    ref, _ = ref_bwd(d, ref_fwd(d)[0])
    rng = np.random.default_rng(0)
    for name, key in (("x", "dx"), ("zr", "dzr"), ("zi", "dzi"), ("lam", "dlam"), ("br", "dbr"), ("bi", "dbi"),
                      ("h0", "dh0")):
        for _ in range(6):
            at = tuple(int(rng.integers(0, n)) for n in d[name].shape)
            e = 1e-5
            up, dn = ({**d, name: d[name].clone()} for _ in range(2))
            up[name][at] += e
            dn[name][at] -= e
            diff = (loss(up) - loss(dn)) / (2 * e)
            assert abs(diff - float(ref[key][at])) <= 1e-7 * max(1.0, abs(diff)), (name, at)


def test_refusals():
    """Argument errors before any device work (CPU)."""
    u, p = torch.zeros(5, 2, 4), torch.zeros(4)
    with pytest.raises(ValueError):
        lrs.glr_fwd(u, u, u, p, p, p)  # host tensors
    with pytest.raises(ValueError):
        lrs.glr_bwd(u, u, u, p, p, p, u, u)
    with pytest.raises(ValueError):
        lrs.glr_step(u[0], u[0], u[0], p, p, p, u[0])
    lib = lrs.load()
    P = None
    assert lib.glr_fwd(*([P] * 10), 2, 3, 4, 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.glr_fwd(*([P] * 10), 2, 3, 4, 5, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.glr_fwd(*([P] * 10), -2, 3, 4, 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.glr_bwd(*([P] * 18), 2, 3, 4, 1, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.glr_step(*([P] * 10), 2, 2, 4, 0, P) == lrs.LR_ERR_INVALID_ARG
    assert lib.glr_step(*([P] * 10), 2, 1, 4, 0, P) == lrs.LR_ERR_INVALID_ARG  # more rows than slots
    assert lib.glr_fwd(*([P] * 10), 1 << 31, 1 << 31, 4, 0, P) == lrs.LR_ERR_TOO_LARGE
    buf = ctypes.create_string_buffer(64)
    odd = ctypes.c_void_p(ctypes.addressof(buf) + 1)
    assert lib.glr_fwd(odd, odd, odd, odd, odd, odd, P, P, odd, P, 1, 1, 1, 0, P) == lrs.LR_ERR_ALIGN
    assert lib.glr_step(odd, odd, odd, odd, odd, odd, P, P, odd, odd, 1, 1, 1, 0, P) == lrs.LR_ERR_ALIGN


@pytest.mark.gpu
def test_refusals_on_device_tensors(cuda):
    d = dev(make(6, 2, 8, "f32"))
    args = [d[k] for k in NAMES]
    for bad in (dict(h0=d["h0"].bfloat16()), dict(h0=d["h0"][:1]), dict(reset=d["reset"][:3]),
                dict(reset=d["reset"].int()), dict(h=torch.empty(6, 2, 8, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            cuda.glr_fwd(*args, **bad)
    with pytest.raises(ValueError):
        cuda.glr_fwd(d["x"].transpose(0, 1), d["zr"], d["zi"], *args[3:])
    with pytest.raises(ValueError):
        cuda.glr_fwd(d["x"], d["zr"].bfloat16(), d["zi"], *args[3:])
    with pytest.raises(ValueError):
        cuda.glr_step(*[a[0].contiguous() if a.dim() == 3 else a for a in args], d["h0"][:1])
    with pytest.raises(TypeError):
        cuda.glr_fwd(*[a.half() if a.dim() == 3 else a for a in args])


def test_shapes_cover_every_plan():
    """The parity shapes above reach one span and several, staged by TMA, through
    registers in vectors and element by element, in both directions (CPU)."""
    for op in ("glr_fwd", "glr_bwd"):
        seen = set()
        for T, B, D in SHAPES:
            for dt in ("f32", "bf16"):
                p = lrs.plan_info(op, dt, D % 4 == 0, T, B * D)
                seen.add((p["protocol"], p["tma"], D % 4 == 0))
        assert seen == {(pr, *kind) for pr in ("chain", "spans")
                        for kind in ((True, True), (False, True), (False, False))}, seen


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("br", [0.0, 3.0, 20.0])
@pytest.mark.parametrize("T,D", [(20, 128), (64, 128), (20, 33)])
def test_input_gates_shut_to_the_last_bit(cuda, T, D, br, dtype):
    """1 + e^-z of the input gate through the range where its reciprocal leaves
    fp32's normal numbers (z about -87.4): the decay beside it stays what it is.
    (The gates are the same at every step, so are the decays' errors: T 1e-7.)"""
    d = make(T, 2, D, dtype, seed=21, resets="none")
    d["zr"][:], d["zi"][:] = 0.0, 0.0
    d["bi"] = torch.linspace(-87.7, -86.5, D)
    d["br"] = torch.full((D,), br)
    c = dev(d)
    h, last = cuda.glr_fwd(*[c[k] for k in NAMES], h0=c["h0"])
    rh, rlast = ref_fwd(d)
    assert err(h, rh) <= TOL[dtype] and err(last, rlast) <= 1e-5


def piece(d, lo, hi):
    """Steps lo .. hi - 1 of a problem, as one that starts and ends without states."""
    cut = {k: v[lo:hi] if k in ("x", "zr", "zi", "dh", "reset") else v for k, v in d.items()}
    return dict(cut, h0=None, dh_last=None)


# one span and several, in vectors by TMA and element by element
RESET_SHAPES = [(20, 128), (300, 128), (20, 33), (300, 33)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("T,D", RESET_SHAPES)
def test_a_reset_drops_a_state_that_is_not_finite(cuda, T, D, bad, dtype):
    """A document whose state overflowed, or an initial state that did, and what a
    reset step's own decay gate holds, reach nothing after the reset."""
    d = make(T, 3, D, dtype, seed=22, resets="none")
    k = T // 2 + 1
    d["reset"] = torch.zeros(T, 3, dtype=torch.uint8)
    d["reset"][k] = 1
    d["h0"][0] = bad
    d["x"][2, 1] = bad
    d["x"][k - 1, 2] = bad
    d["zr"][3, 2, ::3] = bad
    d["zr"][k, :, ::2] = bad
    c = dev(d)
    h, last = cuda.glr_fwd(*[c[n] for n in NAMES], h0=c["h0"], reset=c["reset"])
    clean = dict(d, zr=d["zr"].clone())
    clean["zr"][k] = 0.0
    late = piece(clean, k, T)
    rh, rlast = ref_fwd(late)
    assert not torch.isfinite(h[k - 1]).any()
    assert err(h[k:], rh) <= TOL[dtype] and err(last, rlast) <= 1e-5
    got = cuda.glr_bwd(*[c[n] for n in NAMES], h, c["dh"], h0=c["h0"], reset=c["reset"])
    ref, _ = ref_bwd(late, h[k:].cpu())
    for n in ("dx", "dzr", "dzi"):
        assert err(got[n][k:], ref[n]) <= TOL[dtype], n


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("T,D", RESET_SHAPES)
def test_a_reset_stops_a_gradient_that_is_not_finite(cuda, T, D, bad, dtype):
    """Nothing of a later document's gradient, or of the last state's, reaches the
    steps before its reset."""
    d = make(T, 3, D, dtype, seed=23, resets="none")
    k = T // 2 - 1
    d["reset"] = torch.zeros(T, 3, dtype=torch.uint8)
    d["reset"][k] = 1
    d["dh_last"][0] = bad
    d["dh"][T - 2, 1] = bad
    d["dh"][k, 2] = bad
    c = dev(d)
    args = [c[n] for n in NAMES]
    h, _ = cuda.glr_fwd(*args, h0=c["h0"], reset=c["reset"])
    got = cuda.glr_bwd(*args, h, c["dh"], h0=c["h0"], reset=c["reset"], dh_last=c["dh_last"])
    ref, _ = ref_bwd(dict(piece(d, 0, k), h0=d["h0"]), h[:k].cpu())
    for n in ("dx", "dzr", "dzi"):
        assert err(got[n][:k], ref[n]) <= TOL[dtype], n
    assert err(got["dh0"], ref["dh0"]) <= 1e-5
    assert not torch.isfinite(got["dx"][k, 2]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("with_resets", [False, True])
@pytest.mark.parametrize("T,D", RESET_SHAPES)
def test_a_nan_stays_in_its_document_and_fills_it(cuda, T, D, with_resets):
    """Decays whose products underflow to 0 are no resets: a NaN reaches the end of its
    document (and its gradient the start), over spans and all."""
    d = make(T, 3, D, "f32", seed=24, resets="none")
    d["lam"] = torch.full((D,), 60.0)
    lo, hi, t0 = T // 4, 3 * T // 4, T // 2
    if with_resets:
        d["reset"] = torch.zeros(T, 3, dtype=torch.uint8)
        d["reset"][lo] = d["reset"][hi] = 1
    else:
        lo, hi = 0, T
    d["x"][t0, 1] = float("nan")
    c = dev(d)
    args = [c[n] for n in NAMES]
    h, _ = cuda.glr_fwd(*args, h0=c["h0"], reset=c["reset"])
    bad = torch.zeros(T, 3, dtype=torch.bool)
    bad[t0:hi, 1] = True
    assert torch.equal(torch.isnan(h).cpu(), bad[:, :, None].expand(T, 3, D))
    d["dh"][t0, 2] = float("nan")
    got = cuda.glr_bwd(*args, c["x"].nan_to_num(), d["dh"].cuda(), h0=c["h0"], reset=c["reset"])
    bad = torch.zeros(T, 3, dtype=torch.bool)
    bad[lo:t0 + 1, 2] = True
    # a sequence's own NaN in x shows in its own step only
    assert torch.equal(torch.isnan(got["dx"]).cpu(), bad[:, :, None].expand(T, 3, D))


def test_reset_shapes_are_one_span_and_several():
    for op in ("glr_fwd", "glr_bwd"):
        for dt in ("f32", "bf16"):
            kinds = [lrs.plan_info(op, dt, D % 4 == 0, T, 3 * D) for T, D in RESET_SHAPES]
            assert [p["protocol"] for p in kinds] == ["chain", "spans", "chain", "spans"]
            assert [p["tma"] for p in kinds] == [True, True, False, False]
