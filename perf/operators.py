"""Cases of the operators a recurrent language model trains and decodes with.

Four operators next to the linear-recurrence scan: the gated linear recurrence
(forward, backward, single-token step), layer norm with the residual add
(forward, backward), softmax cross entropy over a large vocabulary without
keeping the logits (loss, gradients) and the AdamW step over many tensors
(moments in 32 or in 8 bits).  `run` computes a case in its plain form
(elementary torch operations in fp32, rounded once at the end) or, with
`own = True`, through the library's calls; `exact` computes it from the
definitions in fp64.
"""
import math

import torch

own = False

IGNORE = -100
BLOCK = 256      # elements that share one scale in the 8-bit moments
RATE_C = 8.0     # the decay rates are -RATE_C log(a) for a base decay a per feature
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of eight sequences whose states sit in a pool of slots: latency
        dict(name="glr_step_bf16_8x1024", op="glr_step", B=8, D=1024, dt="bf16", slots=11, resets=True),
        # a training forward pass over packed documents (a reset at each start), the widest problem
        dict(name="glr_fwd_bf16_8192x16x4096", op="glr_fwd", T=8192, B=16, D=4096, dt="bf16", resets=True),
        # the backward pass of one long, narrow sequence of packed documents
        dict(name="glr_bwd_bf16_65536x1x1024", op="glr_bwd", T=65536, B=1, D=1024, dt="bf16", resets=True),
        # the backward pass of a recurrent layer of 2048 steps by 32 sequences
        dict(name="glr_bwd_f32_2048x32x1024", op="glr_bwd", T=2048, B=32, D=1024, dt="f32", resets=False),
        # the norm before a decode step's projections: a handful of rows, latency
        dict(name="ln_fwd_bf16_8x1024", op="ln_fwd", N=8, D=1024, dt="bf16", res=True),
        # the norm with its residual add over the rows of a training batch
        dict(name="ln_fwd_bf16_131072x4096", op="ln_fwd", N=131072, D=4096, dt="bf16", res=True),
        # its backward pass at an odd width that allows no vector accesses
        dict(name="ln_bwd_f32_30011x1111", op="ln_bwd", N=30011, D=1111, dt="f32", res=False),
        # fp32 fine-tuning on an odd vocabulary with a ragged batch: loss and gradients
        dict(name="lce_train_f32_509x250x10007", op="lce_train", N=509, D=250, V=10007, dt="f32"),
        # the training loss of a language model and its gradients
        dict(name="lce_train_bf16_8192x1024x65536", op="lce_train", N=8192, D=1024, V=65536, dt="bf16"),
        # evaluation: the loss alone over a large vocabulary
        dict(name="lce_loss_bf16_4096x4096x131072", op="lce_loss", N=4096, D=4096, V=131072, dt="bf16"),
        # the optimizer step over a model's tensors, fp32 moments, bf16 gradients and bf16 copies of the weights
        dict(name="adamw_128M", op="adamw", total=128 << 20, tensors=160, gdt="bf16", copies=True, step=100),
        # the same with the moments in 8 bits
        dict(name="adamw8_64M", op="adamw8", total=64 << 20, tensors=90, gdt="f32", copies=False, step=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width over the logarithm of the range: half of them multiples of 128, the rest as they fall."""
    d = _log(rng, lo, hi)
    return max(lo, d // 128 * 128) if rng.random() < 0.5 and d >= 128 else d


def draw(rng):
    op = rng.choice(["glr_step", "glr_fwd", "glr_bwd", "ln_fwd", "ln_bwd", "lce_train", "lce_loss", "adamw", "adamw8"])
    dt = rng.choice(["f32", "bf16"])
    if op == "glr_step":
        B = _log(rng, 1, 512)
        return dict(op=op, B=B, D=_width(rng, 64, 8192), dt=dt, slots=B + rng.randrange(0, 9), resets=rng.random() < 0.5)
    if op in ("glr_fwd", "glr_bwd"):
        n = _log(rng, 1 << 12, 1 << 27)  # elements
        T = _log(rng, 1, min(65536, n // 8))
        D = max(1, min(_width(rng, 8, 4096), n // T))
        return dict(op=op, T=T, B=max(1, min(64, n // (T * D))), D=D, dt=dt, resets=rng.random() < 0.5)
    if op in ("ln_fwd", "ln_bwd"):
        n = _log(rng, 1 << 10, 1 << 28)
        D = min(_width(rng, 16, 16384), n)
        return dict(op=op, N=max(1, n // D), D=D, dt=dt, res=rng.random() < 0.5)
    if op in ("lce_train", "lce_loss"):
        D = _width(rng, 32, 4096)
        V = _width(rng, 100, 131072)
        cap = (40e9 if dt == "f32" else 400e9) / (D * V)
        return dict(op=op, N=_log(rng, 1, max(2, min(8192, cap))), D=D, V=V, dt=dt)
    return dict(op=op, total=_log(rng, 1 << 12, 1 << 26), tensors=rng.randrange(1, 400), gdt=dt,
                copies=rng.random() < 0.5, step=_log(rng, 1, 10000))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _randn(g, shape, dt=torch.float32, std=1.0):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0.0, std, generator=g).to(dt)


def _sizes(case):
    """Tensor sizes of an optimizer case: a few large matrices and many small vectors, odd sizes among them."""
    n, total = case["tensors"], case["total"]
    w = [1.0 / (1 + (i * 7) % n) for i in range(n)]
    scale = total / sum(w)
    return [max(1, int(x * scale) - (i % 3)) for i, x in enumerate(w)]


def _flat(sizes):
    """Offsets of the tensors in one flat buffer, each start a multiple of 64 elements."""
    offs, at = [], 0
    for s in sizes:
        offs.append(at)
        at += (s + 63) // 64 * 64
    return offs, at


def _views(buf, sizes, offs):
    return [buf[o:o + s] for s, o in zip(sizes, offs)]


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case=dict(case))
    if op.startswith("glr"):
        dt, B, D = DT[case["dt"]], case["B"], case["D"]
        shape = (B, D) if op == "glr_step" else (case["T"], B, D)
        for k in ("x", "zr", "zi"):
            s[k] = _randn(g, shape, dt)
        base = torch.empty(D, device="cuda").uniform_(0.9, 0.999, generator=g)
        s["lam"] = -RATE_C * torch.log(base)
        s["br"], s["bi"] = _randn(g, (D,), std=0.5), _randn(g, (D,), std=0.5)
        s["reset"] = None
        if case["resets"]:
            p = 0.1 if op == "glr_step" else min(0.5, 1.0 / 512 + 1.0 / case["T"])
            s["reset"] = (torch.empty(shape[:-1], device="cuda").uniform_(generator=g) < p).to(torch.uint8)
        if op == "glr_step":
            s["state"] = _randn(g, (case["slots"], D))
            # every sequence has a slot of its own; the last row of a larger batch is padding
            s["slots"] = torch.randperm(case["slots"], device="cuda", generator=g)[:B].to(torch.int32)
            if B > 2:
                s["slots"][B - 1] = -1
        else:
            s["h0"] = _randn(g, (B, D))
        if op == "glr_bwd":
            s["dh"] = _randn(g, shape, dt)
            s["dh_last"] = _randn(g, (B, D))
            s["h"] = _plain_glr_fwd(s)[0]
    elif op.startswith("ln"):
        dt, N, D = DT[case["dt"]], case["N"], case["D"]
        s["x"] = _randn(g, (N, D), dt, 1.5) + torch.tensor(0.25, dtype=dt, device="cuda")
        s["w"], s["b"] = 1.0 + _randn(g, (D,), std=0.2), _randn(g, (D,), std=0.2)
        s["res"] = _randn(g, (N, D), dt) if case["res"] else None
        if op == "ln_bwd":
            s["dy"] = _randn(g, (N, D), dt)
            s["mean"], s["rstd"] = _plain_stats(s["x"].float())
    elif op.startswith("lce"):
        dt, N, D, V = DT[case["dt"]], case["N"], case["D"], case["V"]
        s["x"] = _randn(g, (N, D), dt)
        s["w"] = _randn(g, (V, D), dt, 2.0 / math.sqrt(D))
        t = torch.randint(0, V, (N,), device="cuda", generator=g)
        pad = torch.empty(N, device="cuda").uniform_(generator=g) < 0.1  # padding tokens
        s["target"] = torch.where(pad, torch.full_like(t, IGNORE), t)
        # the mean over the tokens that count
        s["dloss"] = (1.0 / (~pad).sum().clamp(min=1).float()).expand(N).contiguous()
    else:
        sizes = _sizes(case)
        offs, n = _flat(sizes)
        s["sizes"], s["offs"], s["n"] = sizes, offs, n
        s["p"] = _randn(g, (n,), std=0.02)
        s["g"] = _randn(g, (n,), DT[case["gdt"]], 1e-3)
        s["copy"] = torch.zeros(n, device="cuda", dtype=torch.bfloat16) if case["copies"] else None
        s["scale"] = torch.empty(1, device="cuda").uniform_(0.5, 1.0, generator=g)  # gradient clipping's factor
        m = _randn(g, (n,), std=1e-3)
        v = _randn(g, (n,), std=1e-3).square() + 1e-9
        s["seed"] = 12345 + seed
        if op == "adamw":
            s["m"], s["v"] = m, v
        else:
            nb = (n + BLOCK - 1) // BLOCK
            s["boffs"] = []
            at = 0
            for z in sizes:
                s["boffs"].append(at)
                at += (z + BLOCK - 1) // BLOCK
            s["mq"] = torch.zeros(n, device="cuda", dtype=torch.int8)
            s["vq"] = torch.zeros(n, device="cuda", dtype=torch.uint8)
            s["ms"], s["vs"] = torch.zeros(at, device="cuda"), torch.zeros(at, device="cuda")
            for i, (z, o, bo) in enumerate(zip(sizes, offs, s["boffs"])):
                mq, ms = _encode_m(m[o:o + z], torch.full((z,), 0.5, device="cuda"))
                vq, vs = _encode_v(v[o:o + z], torch.full((z,), 0.5, device="cuda"))
                s["mq"][o:o + z], s["vq"][o:o + z] = mq, vq
                s["ms"][bo:bo + ms.numel()], s["vs"][bo:bo + vs.numel()] = ms, vs
            del nb
        lists = {k: _views(s[k], sizes, offs) for k in ("p", "g", "m", "v", "mq", "vq") if k in s}
        if s["copy"] is not None:
            lists["copy"] = _views(s["copy"], sizes, offs)
        if op == "adamw8":
            nbs = [(z + BLOCK - 1) // BLOCK for z in sizes]
            lists["ms"], lists["vs"] = _views(s["ms"], nbs, s["boffs"]), _views(s["vs"], nbs, s["boffs"])
            s["mval"], s["vval"] = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
            lists["mval"], lists["vval"] = _views(s["mval"], sizes, offs), _views(s["vval"], sizes, offs)
        s["lists"] = lists
    return s


HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


# ------------------------------------------------------------- plain forms

def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _gates(s):
    """r, i, the decay a, its square a2 and the input's factor sqrt(1 - a2); a reset row has a = 0."""
    r = _sigmoid(s["zr"].float() + s["br"])
    i = _sigmoid(s["zi"].float() + s["bi"])
    la = -s["lam"] * r
    a = torch.exp(la)
    f = torch.sqrt(-torch.expm1(2.0 * la))
    if s["reset"] is not None:
        k = (s["reset"] != 0).unsqueeze(-1)
        a, f = a.masked_fill(k, 0.0), f.masked_fill(k, 1.0)
    return r, i, a, f


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 0 in log2(T) passes; both arguments are used up."""
    off, T = 1, a.shape[0]
    while off < T:
        b[off:] += a[off:] * b[:-off].clone()
        a[off:] *= a[:-off].clone()
        off *= 2
    return b


def _plain_glr_fwd(s):
    r, i, a, f = _gates(s)
    b = f * i * s["x"].float()
    b[0] += a[0] * s["h0"]
    h = _scan(a, b)
    return h.to(s["x"].dtype), h[-1].clone()


def _plain_glr_bwd(s):
    x = s["x"].float()
    r, i, a, f = _gates(s)
    hp = torch.cat([s["h0"].unsqueeze(0), s["h"][:-1].float()])
    # delta_t = dh_t + a_{t+1} delta_{t+1}, the scan in reverse time
    d = s["dh"].float().clone()
    d[-1] += s["dh_last"]
    an = torch.zeros_like(a)
    an[:-1] = a[1:]
    d = _scan(an.flip(0), d.flip(0)).flip(0)
    u = i * x
    keep = f > 0.0  # no gradient of the decay where it is 1 to the last bit
    if s["reset"] is not None:
        keep = keep & (s["reset"] == 0).unsqueeze(-1)
    dla = torch.where(keep, d * (a * hp - u * (a * a) / torch.where(keep, f, torch.ones_like(f))), torch.zeros_like(d))
    du = d * f
    dzr = -s["lam"] * dla * r * (1.0 - r)
    dzi = du * x * i * (1.0 - i)
    dt = s["x"].dtype
    return dict(dx=(du * i).to(dt), dzr=dzr.to(dt), dzi=dzi.to(dt), dlam=-(dla * r).sum((0, 1)),
                dbr=dzr.sum((0, 1)), dbi=dzi.sum((0, 1)), dh0=a[0] * d[0])


def _plain_glr_step(s):
    r, i, a, f = _gates(s)
    live, n = s["slots"] >= 0, s["state"].shape[0]
    at = torch.where(live, s["slots"], torch.full_like(s["slots"], n)).long()
    pool = torch.cat([s["state"], torch.zeros_like(s["state"][:1])])  # one row more, for the padding
    h = a * pool[at] + f * i * s["x"].float()
    pool[at] = h
    s["state"].copy_(pool[:n])
    return (h * live.unsqueeze(-1)).to(s["x"].dtype), s["state"]


EPS = 1e-5


def _plain_stats(x):
    mean = x.mean(-1)
    c = x - mean.unsqueeze(-1)
    return mean, 1.0 / torch.sqrt((c * c).mean(-1) + EPS)


def _plain_ln_fwd(s):
    dt = s["x"].dtype
    x = s["x"].float()
    if s["res"] is not None:
        x = (x + s["res"].float()).to(dt).float()  # the sum is an output of its own; the norm is taken of what is kept
    mean, rstd = _plain_stats(x)
    y = (x - mean.unsqueeze(-1)) * rstd.unsqueeze(-1) * s["w"] + s["b"]
    return dict(y=y.to(dt), mean=mean, rstd=rstd, **({"s": x.to(dt)} if s["res"] is not None else {}))


def _plain_ln_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"].unsqueeze(-1)) * s["rstd"].unsqueeze(-1)
    t = dy * s["w"]
    dx = (t - t.mean(-1, keepdim=True) - xh * (t * xh).mean(-1, keepdim=True)) * s["rstd"].unsqueeze(-1)
    if s["res"] is not None:
        dx = dx + s["res"].float()  # the gradient that the residual stream brings
    return dict(dx=dx.to(s["x"].dtype), dw=(dy * xh).sum(0), db=dy.sum(0))


def _plain_lce(s, train):
    x, w = s["x"].float(), s["w"].float()
    l = x @ w.t()
    live = s["target"] != IGNORE
    t = torch.where(live, s["target"], torch.zeros_like(s["target"]))
    top = l.max(-1).values
    lt = l[torch.arange(l.shape[0], device=l.device), t]
    l = torch.exp(l - top.unsqueeze(-1))
    z = l.sum(-1)
    lse = top + torch.log(z)
    loss = torch.where(live, lse - lt, torch.zeros_like(lse))
    if not train:
        return dict(loss=loss, lse=lse)
    l /= z.unsqueeze(-1)
    l[torch.arange(l.shape[0], device=l.device), t] -= 1.0
    l *= torch.where(live, s["dloss"], torch.zeros_like(s["dloss"])).unsqueeze(-1)
    return dict(loss=loss, lse=lse, dx=(l @ w).to(s["x"].dtype), dw=(l.t() @ x).to(s["w"].dtype))


# 8-bit moments: blocks of 256 elements share a scale, the largest magnitude;
# m = scale sign(q) (q/127)^2, v = scale (q/255)^4, rounded up or down with the
# probability that keeps the rooted value right in the mean.

def _noise(n, seed, tensor):
    """16 random bits for m and 16 for v of every element, a hash of its index, the tensor's and the step's seed."""
    M = 0xFFFFFFFF
    h = (torch.arange(n, device="cuda", dtype=torch.int64) + tensor * 0x9E3779B1 + seed * 0xBB67AE85) & M
    h = ((h ^ (h >> 16)) * 0x6A09E667) & M  # the fractional bits of the roots of 3, 2 and 5, made odd
    h = ((h ^ (h >> 15)) * 0x3C6EF373) & M
    h = h ^ (h >> 16)
    return (h >> 16).float() * 2.0 ** -16, (h & 0xFFFF).float() * 2.0 ** -16


def _blocks(x):
    n = x.numel()
    nb = (n + BLOCK - 1) // BLOCK
    p = torch.zeros(nb * BLOCK, device=x.device)
    p[:n] = x
    return p.view(nb, BLOCK)


def _ratio(x):
    b = _blocks(x.abs())
    scale = b.max(-1).values
    inv = torch.where(scale > 0, torch.reciprocal(scale), torch.zeros_like(scale))
    return (b * inv.unsqueeze(-1)).view(-1)[:x.numel()], scale


def _encode_m(m, u):
    r, scale = _ratio(m)
    q = torch.floor(torch.sqrt(r) * 127.0 + u).clamp(max=127.0)
    return torch.where(m < 0, -q, q).to(torch.int8), scale


def _encode_v(v, u):
    r, scale = _ratio(v)
    q = torch.floor(torch.sqrt(torch.sqrt(r)) * 255.0 + u).clamp(max=255.0)
    q = torch.where((v > 0) & (q < 1.0), torch.ones_like(q), q)  # no positive v becomes 0: the step divides by its root
    return q.to(torch.uint8), scale


def _spread(scale, n):
    return scale.repeat_interleave(BLOCK)[:n]


def _decode_m(q, scale):
    t = q.float() * (1.0 / 127.0)
    return (t * t.abs()) * _spread(scale, q.numel())


def _decode_v(q, scale):
    t = q.float() * (1.0 / 255.0)
    t = t * t
    return (t * t) * _spread(scale, q.numel())


def _plain_adamw(s):
    c, L, h = s["case"], s["lists"], HYPER
    k1, k2 = 1.0 - h["beta1"] ** c["step"], 1.0 - h["beta2"] ** c["step"]
    eight = c["op"] == "adamw8"
    for i in range(len(s["sizes"])):
        p, g = L["p"][i], L["g"][i].float() * s["scale"]
        if eight:
            m, v = _decode_m(L["mq"][i], L["ms"][i]), _decode_v(L["vq"][i], L["vs"][i])
        else:
            m, v = L["m"][i], L["v"][i]
        m = h["beta1"] * m + (1.0 - h["beta1"]) * g
        v = h["beta2"] * v + (1.0 - h["beta2"]) * (g * g)
        p.copy_(p * (1.0 - h["lr"] * h["weight_decay"]) - h["lr"] * (m / k1) / (torch.sqrt(v / k2) + h["eps"]))
        if c["copies"]:
            L["copy"][i].copy_(p)
        if eight:
            um, uv = _noise(p.numel(), s["seed"], i)
            mq, ms = _encode_m(m, um)
            vq, vs = _encode_v(v, uv)
            for to, x in ((L["mq"][i], mq), (L["ms"][i], ms), (L["vq"][i], vq), (L["vs"][i], vs)):
                to.copy_(x)
            L["mval"][i].copy_(_decode_m(mq, ms))
            L["vval"][i].copy_(_decode_v(vq, vs))
        else:
            L["m"][i].copy_(m)
            L["v"][i].copy_(v)
    return _adamw_out(s)


def _adamw_out(s):
    eight = s["case"]["op"] == "adamw8"
    r = dict(p=s["p"], m=s["mval"] if eight else s["m"], v=s["vval"] if eight else s["v"])
    if s["copy"] is not None:
        r["copy"] = s["copy"]
    return r


# --------------------------------------------------------------------- run

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _own(s, op)
    if op == "glr_fwd":
        h, last = _plain_glr_fwd(s)
        return dict(h=h, h_last=last)
    if op == "glr_bwd":
        return _plain_glr_bwd(s)
    if op == "glr_step":
        h, pool = _plain_glr_step(s)
        return dict(h=h, state=pool)
    if op == "ln_fwd":
        return _plain_ln_fwd(s)
    if op == "ln_bwd":
        return _plain_ln_bwd(s)
    if op.startswith("lce"):
        return _plain_lce(s, op == "lce_train")
    return _plain_adamw(s)


def _own(s, op):
    import linear_recurrence_scan_chunked_gb300 as lrs
    c = s["case"]
    if op == "glr_fwd":
        h, last = lrs.glr_fwd(s["x"], s["zr"], s["zi"], s["lam"], s["br"], s["bi"], h0=s["h0"], reset=s["reset"])
        return dict(h=h, h_last=last)
    if op == "glr_bwd":
        return lrs.glr_bwd(s["x"], s["zr"], s["zi"], s["lam"], s["br"], s["bi"], s["h"], s["dh"], h0=s["h0"],
                           reset=s["reset"], dh_last=s["dh_last"])
    if op == "glr_step":
        h = lrs.glr_step(s["x"], s["zr"], s["zi"], s["lam"], s["br"], s["bi"], s["state"], slots=s["slots"],
                         reset=s["reset"])
        return dict(h=h, state=s["state"])
    if op == "ln_fwd":
        r = lrs.layer_norm_fwd(s["x"], s["w"], s["b"], res=s["res"], eps=EPS)
        return dict(zip(("y", "mean", "rstd", "s"), r))
    if op == "ln_bwd":
        return lrs.layer_norm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["dy"], dres=s["res"])
    if op.startswith("lce"):
        loss, lse = lrs.lce_fwd(s["x"], s["w"], s["target"], ignore=IGNORE)
        if op == "lce_loss":
            return dict(loss=loss, lse=lse)
        dx, dw = lrs.lce_bwd(s["x"], s["w"], s["target"], lse, s["dloss"], ignore=IGNORE)
        return dict(loss=loss, lse=lse, dx=dx, dw=dw)
    L = s["lists"]
    if op == "adamw":
        lrs.adamw_step(L["p"], L["g"], L["m"], L["v"], step=c["step"], grad_scale=s["scale"],
                       copies=L.get("copy"), **HYPER)
    else:
        lrs.adamw8_step(L["p"], L["g"], L["mq"], L["vq"], L["ms"], L["vs"], step=c["step"], seed=s["seed"],
                        grad_scale=s["scale"], copies=L.get("copy"), **HYPER)
        lrs.adamw8_values(L["mq"], L["vq"], L["ms"], L["vs"], m=L["mval"], v=L["vval"])
    return _adamw_out(s)


# -------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op.startswith("glr"):
        es = 4 if case["dt"] == "f32" else 2
        BD = case["B"] * case["D"]
        if op == "glr_step":  # three inputs, one output, the state read and written
            live = case["B"] - 1 if case["B"] > 2 else case["B"]
            return dict(bytes=BD * 4 * es + live * case["D"] * 8, flops=20 * BD)
        n = case["T"] * BD
        arrays = 4 if op == "glr_fwd" else 8
        extra = 8 * BD + (case["T"] * case["B"] if case["resets"] else 0) + 12 * case["D"]
        return dict(bytes=n * arrays * es + extra, flops=n * (20 if op == "glr_fwd" else 50))
    if op.startswith("ln"):
        es, n = 4 if case["dt"] == "f32" else 2, case["N"] * case["D"]
        arrays = (4 if case["res"] else 2) if op == "ln_fwd" else (4 if case["res"] else 3)
        return dict(bytes=n * arrays * es + 8 * case["N"] + 8 * case["D"], flops=n * (8 if op == "ln_fwd" else 14))
    if op.startswith("lce"):
        es = 4 if case["dt"] == "f32" else 2
        N, D, V = case["N"], case["D"], case["V"]
        k = 2 if op == "lce_train" else 1
        return dict(bytes=k * (N + V) * D * es + 16 * N, flops=(6 if op == "lce_train" else 2) * N * D * V)
    n = sum(_sizes(case))
    g = 2 if case["gdt"] == "bf16" else 4
    state = 16 if op == "adamw" else 4 + 8  # 8 bits: codes read and written, and the values handed out
    return dict(bytes=n * (8 + g + state + (2 if case["copies"] else 0)), flops=n * 20)


# ------------------------------------------------------------------- exact

def exact(case, seed):
    op = case["op"]
    if op.startswith("lce") and 2.0 * case["N"] * case["D"] * case["V"] * (3 if op == "lce_train" else 1) > 8e12:
        return None
    s = prepare(case, seed)
    if op.startswith("glr"):
        return _exact_glr(s, op)
    if op.startswith("ln"):
        return _exact_ln(s, op)
    if op.startswith("lce"):
        return _exact_lce(s, op)
    return _exact_adamw(s, case)


def _exact_glr(s, op):
    D64 = torch.float64
    lam, br, bi, x = (s[k].to(D64) for k in ("lam", "br", "bi", "x"))
    r = torch.sigmoid(s["zr"].to(D64) + br)
    i = torch.sigmoid(s["zi"].to(D64) + bi)
    a = torch.exp(-lam * r)
    f = torch.sqrt(-torch.expm1(-2.0 * lam * r))
    if s["reset"] is not None:
        a[s["reset"] != 0] = 0.0
        f[s["reset"] != 0] = 1.0
    b = f * i * x
    if op == "glr_step":
        pool, out = s["state"].to(D64), torch.zeros_like(x)
        for row, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                out[row] = pool[slot] = a[row] * pool[slot] + b[row]
        return dict(h=out, state=pool)
    T = x.shape[0]
    if op == "glr_fwd":
        h = s["h0"].to(D64)
        for t in range(T):  # the recurrence, step by step; b becomes h
            h = torch.addcmul(b[t], a[t], h, out=b[t])
        return dict(h=b, h_last=h)
    # what the step after t passes back is a_{t+1} d_{t+1}; dh becomes d
    d = s["dh"].to(D64)
    d[-1] += s["dh_last"]
    for t in range(T - 2, -1, -1):
        d[t].addcmul_(a[t + 1], d[t + 1])
    dh0 = a[0] * d[0]
    hp = torch.cat([s["h0"].to(D64)[None], s["h"][:-1].to(D64)])
    # h = a hp + f i x with a = exp(-lam r) and f = sqrt(1 - a a): df/da = -a / f
    da = d * (hp - i * x * a / f)
    if s["reset"] is not None:
        da[s["reset"] != 0] = 0.0
    dlam = -(r * a * da).sum((0, 1))
    dzr = -lam * a * da * r * (1.0 - r)
    dzi = d * b * (1.0 - i)
    return dict(dx=d * f * i, dzr=dzr, dzi=dzi, dlam=dlam, dbr=dzr.sum((0, 1)), dbi=dzi.sum((0, 1)), dh0=dh0)


def _exact_ln(s, op):
    x = s["x"].double()
    N, D = x.shape
    step = max(1, (1 << 27) // D)
    if op == "ln_fwd":
        y, mean, rstd, kept = [], [], [], []
        for lo in range(0, N, step):
            z = x[lo:lo + step]
            if s["res"] is not None:
                z = z + s["res"][lo:lo + step].double()
                kept.append(z)
                z = z.float().to(s["x"].dtype).double()  # the sum as it is kept
            var, mu = torch.var_mean(z, -1, correction=0)
            mean.append(mu)
            rstd.append((var + EPS).rsqrt())
            y.append((z - mu[:, None]) * rstd[-1][:, None] * s["w"].double() + s["b"].double())
        r = dict(y=torch.cat(y), mean=torch.cat(mean), rstd=torch.cat(rstd))
        return dict(r, s=torch.cat(kept)) if kept else r
    dw, db, dx = torch.zeros(D, device="cuda", dtype=torch.float64), torch.zeros(D, device="cuda", dtype=torch.float64), []
    for lo in range(0, N, step):
        z, dy = x[lo:lo + step], s["dy"][lo:lo + step].double()
        mu, rs = s["mean"][lo:lo + step].double()[:, None], s["rstd"][lo:lo + step].double()[:, None]
        xh = (z - mu) * rs
        dw += (dy * xh).sum(0)
        db += dy.sum(0)
        t = dy * s["w"].double()
        a = torch.linalg.vecdot(t, xh)[:, None] / D
        q = rs * (t - xh * a - t.sum(-1, keepdim=True) / D)
        dx.append(q + s["res"][lo:lo + step].double() if s["res"] is not None else q)
    return dict(dx=torch.cat(dx), dw=dw, db=db)


def _exact_lce(s, op):
    w = s["w"].double()
    N, V = s["x"].shape[0], w.shape[0]
    step = max(1, (1 << 27) // V)
    loss, lse, dx, dw = [], [], [], torch.zeros_like(w) if op == "lce_train" else None
    for lo in range(0, N, step):
        x, t = s["x"][lo:lo + step].double(), s["target"][lo:lo + step]
        logit = torch.mm(x, w.T)
        live = t.ne(IGNORE)
        z = torch.logsumexp(logit, 1)
        lse.append(z)
        at = t.clamp(min=0)[:, None]
        loss.append((z - logit.gather(1, at)[:, 0]) * live)
        if op == "lce_train":
            p = torch.softmax(logit, 1).scatter_add_(1, at, -torch.ones(at.shape, device="cuda", dtype=torch.float64))
            p *= (s["dloss"][lo:lo + step].double() * live)[:, None]
            dx.append(torch.mm(p, w))
            dw.addmm_(p.T, x)
    r = dict(loss=torch.cat(loss), lse=torch.cat(lse))
    return dict(r, dx=torch.cat(dx), dw=dw) if op == "lce_train" else r


def _exact_adamw(s, case):
    h, eight = HYPER, case["op"] == "adamw8"
    out = {k: s["p"].double().clone() if k == "p" else torch.zeros(s["n"], device="cuda", dtype=torch.float64)
           for k in ("p", "m", "v")}
    if not eight:
        out["m"].copy_(s["m"])
        out["v"].copy_(s["v"])
    for i, (n, o) in enumerate(zip(s["sizes"], s["offs"])):
        grad = s["g"][o:o + n].double() * s["scale"].double()
        if eight:
            blk = torch.arange(n, device="cuda") // BLOCK + s["boffs"][i]
            q = s["mq"][o:o + n].double() / 127
            m = q.sign() * q.square() * s["ms"].double()[blk]
            v = (s["vq"][o:o + n].double() / 255).pow(4) * s["vs"].double()[blk]
        else:
            m, v = s["m"][o:o + n].double(), s["v"][o:o + n].double()
        m = torch.lerp(grad, m, h["beta1"])
        v = torch.lerp(grad.square(), v, h["beta2"])
        mh, vh = m / (1 - h["beta1"] ** case["step"]), v / (1 - h["beta2"] ** case["step"])
        p = out["p"][o:o + n]
        p -= h["lr"] * (mh / (vh.sqrt() + h["eps"]) + h["weight_decay"] * p)
        out["m"][o:o + n], out["v"][o:o + n] = m, v
    r = dict(p=out["p"], m=None if eight else out["m"], v=None if eight else out["v"])
    if case["copies"]:
        copy = torch.zeros_like(out["p"])
        for n, o in zip(s["sizes"], s["offs"]):
            copy[o:o + n] = out["p"][o:o + n]
        r["copy"] = copy
    return r
