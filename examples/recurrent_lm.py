"""A recurrent language model on the library: training steps and decoding.

Embedding, L blocks (layer norm, three projections, the gated linear
recurrence, an output projection, residual stream), a last norm and the
vocabulary cross entropy; AdamW with moments in 32 or 8 bits.  The library does
the norms, the recurrence, the loss and the optimizer; PyTorch the matrix
products and the embedding.  Sequences are [T, B, D] like everywhere in the
library; a step of a document's first token carries a reset, so that documents
can be packed one after the other.

    python examples/recurrent_lm.py            # trains on synthetic text, then decodes
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import linear_recurrence_scan_chunked_gb300 as lrs  # noqa: E402

IGNORE = -100
RATE = 8.0  # decay rates are RATE * softplus(raw)


class RecurrentLM:
    """Parameters (fp32, with copies of the storage type for the products) and
    the forward, backward and decoding passes, written out."""

    def __init__(self, vocab, width, layers, dtype=torch.bfloat16, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s, std: (std * torch.randn(*s, generator=g)).to(device)
        self.vocab, self.width, self.layers, self.dtype = vocab, width, layers, dtype
        p = {"emb": rn(vocab, width, std=1.0), "head": rn(vocab, width, std=width ** -0.5)}
        for i in range(layers + 1):
            p[f"ln{i}.w"] = torch.ones(width, device=device)
            p[f"ln{i}.b"] = torch.zeros(width, device=device)
        for i in range(layers):
            for k in ("x", "zr", "zi", "o"):
                p[f"{i}.W{k}"] = rn(width, width, std=width ** -0.5)
            # decays from 0.9 to 0.999 at an open gate
            base = 0.9 + 0.099 * torch.rand(width, generator=g).to(device)
            p[f"{i}.rate"] = torch.log(torch.expm1(-torch.log(base)))
            p[f"{i}.br"] = torch.zeros(width, device=device)
            p[f"{i}.bi"] = torch.zeros(width, device=device)
        self.p = p
        self.c = {k: v.to(dtype) for k, v in p.items()}  # what the products read

    def lam(self, i):
        return RATE * torch.nn.functional.softplus(self.p[f"{i}.rate"])

    def forward(self, tokens, target, reset=None, states=None):
        """tokens, target [T, B] -> (loss per token [T, B], what backward needs).
        states: a list of [B, D] fp32 states to start from, one per block."""
        keep, T = [], self.c
        s = T["emb"][tokens]
        y, mean, rstd = lrs.layer_norm_fwd(s, self.p["ln0.w"], self.p["ln0.b"])
        last = []
        for i in range(self.layers):
            u, zr, zi = (y @ T[f"{i}.W{k}"] for k in ("x", "zr", "zi"))
            lam = self.lam(i)
            h0 = None if states is None else states[i]
            h, end = lrs.glr_fwd(u, zr, zi, lam, self.p[f"{i}.br"], self.p[f"{i}.bi"], h0=h0, reset=reset)
            last.append(end)
            o = h @ T[f"{i}.Wo"]
            keep.append((s, y, mean, rstd, u, zr, zi, lam, h0, h))
            y, mean, rstd, s = lrs.layer_norm_fwd(o, self.p[f"ln{i + 1}.w"], self.p[f"ln{i + 1}.b"], res=s)
        loss, lse = lrs.lce_fwd(y, T["head"], target, ignore=IGNORE)
        return loss, dict(keep=keep, end=(s, y, mean, rstd), lse=lse, tokens=tokens, target=target, reset=reset,
                          states=last)

    def backward(self, ctx, dloss):
        """Gradients of sum(dloss * loss) for every parameter, dloss [T, B] fp32."""
        g, T = {}, self.c
        s, y, mean, rstd = ctx["end"]
        dy, g["head"] = lrs.lce_bwd(y, T["head"], ctx["target"], ctx["lse"], dloss, ignore=IGNORE)
        ds = None
        for i in range(self.layers, -1, -1):
            r = lrs.layer_norm_bwd(s, self.p[f"ln{i}.w"], mean, rstd, dy, dres=ds)
            ds, g[f"ln{i}.w"], g[f"ln{i}.b"] = r["dx"], r["dw"], r["db"]
            if i == 0:
                break
            j = i - 1
            s, y, mean, rstd, u, zr, zi, lam, h0, h = ctx["keep"][j]
            flat = lambda t: t.reshape(-1, self.width)
            g[f"{j}.Wo"] = flat(h).t() @ flat(ds)
            r = lrs.glr_bwd(u, zr, zi, lam, self.p[f"{j}.br"], self.p[f"{j}.bi"], h, ds @ T[f"{j}.Wo"].t(), h0=h0,
                            reset=ctx["reset"], want_dh0=False)
            g[f"{j}.rate"] = r["dlam"] * RATE * torch.sigmoid(self.p[f"{j}.rate"])
            g[f"{j}.br"], g[f"{j}.bi"] = r["dbr"], r["dbi"]
            dy = 0
            for k, d in (("x", r["dx"]), ("zr", r["dzr"]), ("zi", r["dzi"])):
                g[f"{j}.W{k}"] = flat(y).t() @ flat(d)
                dy = dy + d @ T[f"{j}.W{k}"].t()
        g["emb"] = torch.zeros_like(self.p["emb"]).index_add_(0, ctx["tokens"].reshape(-1), flat(ds).float())
        return g

    def decode(self, tokens, pools, slots, reset=None):
        """One token of each sequence: tokens [B] -> logits [B, V]; pools: one fp32
        state pool [n_slots, D] per block, updated in place."""
        T = self.c
        s = T["emb"][tokens]
        y, _, _ = lrs.layer_norm_fwd(s, self.p["ln0.w"], self.p["ln0.b"])
        for i in range(self.layers):
            u, zr, zi = (y @ T[f"{i}.W{k}"] for k in ("x", "zr", "zi"))
            h = lrs.glr_step(u, zr, zi, self.lam(i), self.p[f"{i}.br"], self.p[f"{i}.bi"], pools[i], slots=slots, reset=reset)
            y, _, _, s = lrs.layer_norm_fwd(h @ T[f"{i}.Wo"], self.p[f"ln{i + 1}.w"], self.p[f"ln{i + 1}.b"], res=s)
        return y.float() @ T["head"].float().t()


class Optimizer:
    """AdamW over the model's parameters with gradient clipping, moments in 32 or 8 bits."""

    def __init__(self, model, lr=3e-3, bits=32, clip=1.0):
        self.m, self.lr, self.bits, self.clip, self.t = model, lr, bits, clip, 0
        self.names = sorted(model.p)
        ps = [model.p[k] for k in self.names]
        self.state = lrs.adamw8_state(ps) if bits == 8 else ([torch.zeros_like(p) for p in ps], [torch.zeros_like(p) for p in ps])

    def step(self, grads):
        self.t += 1
        model = self.m
        # the library takes gradients of one type: the vectors' are fp32, the matrices' of the storage type
        g = [grads[k].float().contiguous() for k in self.names]
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(x) for x in g]))
        scale = (self.clip / (norm + 1e-6)).clamp(max=1.0).reshape(1)
        ps = [model.p[k] for k in self.names]
        copies = [model.c[k] for k in self.names] if model.dtype == torch.bfloat16 else None
        kw = dict(step=self.t, lr=self.lr, beta1=0.9, beta2=0.95, weight_decay=0.01, grad_scale=scale, copies=copies)
        if self.bits == 8:
            lrs.adamw8_step(ps, g, *self.state, seed=self.t, **kw)
        else:
            lrs.adamw_step(ps, g, *self.state, **kw)
        if copies is None:
            for k in self.names:
                model.c[k].copy_(model.p[k])
        return norm


def synthetic(vocab, T, B, gen, device="cuda"):
    """Packed documents in which every token follows from the one before (plus 1
    or times 2, by the document): a batch of (tokens, targets, resets)."""
    tok = torch.empty(T + 1, B, dtype=torch.int64)
    start = torch.zeros(T + 1, B, dtype=torch.uint8)
    for b in range(B):
        t = 0
        while t <= T:
            n = int(torch.randint(8, 40, (1,), generator=gen))
            x, add = int(torch.randint(0, vocab, (1,), generator=gen)), int(torch.randint(0, 2, (1,), generator=gen))
            start[t, b] = 1
            for _ in range(n):
                if t > T:
                    break
                tok[t, b] = x
                x = (x + 1) % vocab if add else (2 * x + 1) % vocab
                t += 1
    target = tok[1:].clone()
    target[start[1:].bool()] = IGNORE  # a document's first token follows from nothing
    reset = start[:T].contiguous()
    return tok[:T].contiguous().to(device), target.to(device), reset.to(device)


def train_step(model, opt, batch):
    tokens, target, reset = batch
    loss, ctx = model.forward(tokens, target, reset)
    live = (target != IGNORE).sum().clamp(min=1).float()
    grads = model.backward(ctx, (1.0 / live).expand(target.shape).contiguous())
    opt.step(grads)
    return loss.sum() / live


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--vocab", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=150)
    ap.add_argument("--bits", type=int, default=32, choices=(32, 8), help="of the optimizer's moments")
    ap.add_argument("--dtype", default="bf16", choices=("bf16", "f32"))
    a = ap.parse_args()
    gen = torch.Generator().manual_seed(1)
    model = RecurrentLM(a.vocab, a.width, a.layers, torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    opt = Optimizer(model, bits=a.bits)
    for i in range(a.steps):
        loss = train_step(model, opt, synthetic(a.vocab, 128, 16, gen))
        if i % 25 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {float(loss):.3f}")
    tokens, _, _ = synthetic(a.vocab, 12, 3, gen)
    pools = [torch.zeros(3, a.width, device="cuda") for _ in range(a.layers)]
    slots = torch.arange(3, dtype=torch.int32, device="cuda")
    for t in range(12):
        nxt = model.decode(tokens[t], pools, slots).argmax(-1)
    out = [nxt]
    for _ in range(8):
        out.append(model.decode(out[-1], pools, slots).argmax(-1))
    print("prompts      ", tokens.t().tolist())
    print("continuations", torch.stack(out, 1).tolist())
    if lrs.last_error() != lrs.LR_OK:
        raise SystemExit("device error word set")


if __name__ == "__main__":
    main()
