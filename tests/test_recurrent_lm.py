"""The operators together, as examples/recurrent_lm.py runs them: the written-out
gradients against fp64 automatic differentiation of the same model, decoding
against the sequence form, and training that learns."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("recurrent_lm", os.path.join(ROOT, "examples", "recurrent_lm.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(lm, p, layers, tokens, target, reset):
    """The model in fp64 on plain tensor operations (CPU), for autograd."""
    def norm(x, w, b):
        mu = x.mean(-1, keepdim=True)
        return (x - mu) / ((x - mu).square().mean(-1, keepdim=True) + 1e-5).sqrt() * w + b

    s = p["emb"][tokens]
    y = norm(s, p["ln0.w"], p["ln0.b"])
    for i in range(layers):
        u, zr, zi = (y @ p[f"{i}.W{k}"] for k in ("x", "zr", "zi"))
        lam = lm.RATE * torch.nn.functional.softplus(p[f"{i}.rate"])
        a = torch.exp(-lam * torch.sigmoid(zr + p[f"{i}.br"]))
        b = torch.sigmoid(zi + p[f"{i}.bi"]) * u
        k = (reset != 0)[..., None]
        f = torch.where(k, 1.0, torch.sqrt(1 - a * a))
        a = torch.where(k, 0.0, a)
        h, hs = torch.zeros_like(s[0]), []
        for t in range(s.shape[0]):
            h = a[t] * h + f[t] * b[t]
            hs.append(h)
        s = s + torch.stack(hs) @ p[f"{i}.Wo"]
        y = norm(s, p[f"ln{i + 1}.w"], p[f"ln{i + 1}.b"])
    l = y @ p["head"].T
    live = target != lm.IGNORE
    nll = -torch.log_softmax(l, -1).gather(-1, target.clamp(min=0)[..., None])[..., 0]
    return torch.where(live, nll, 0.0)


@pytest.mark.gpu
def test_gradients_of_the_whole_model(cuda, lm):
    """fp32 storage: every gradient within 1e-4 of its norm (chains of about ten
    products of 48 terms at 6e-8 each, and the norms' and gates' amplification)."""
    gen = torch.Generator().manual_seed(3)
    model = lm.RecurrentLM(97, 48, 2, torch.float32, seed=5)
    tokens, target, reset = lm.synthetic(97, 37, 3, gen)
    dloss = torch.rand(37, 3, generator=gen).cuda() / 100
    loss, ctx = model.forward(tokens, target, reset)
    grads = model.backward(ctx, dloss)
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in model.p.items()}
    ref = reference(lm, p, 2, tokens.cpu(), target.cpu(), reset.cpu())
    assert float((loss.double().cpu() - ref.detach()).abs().max()) <= 1e-4
    (ref * dloss.double().cpu()).sum().backward()
    assert set(grads) == set(p)
    for k in p:
        n = float(p[k].grad.norm())
        assert float((grads[k].double().cpu() - p[k].grad).norm()) <= 1e-4 * n + 1e-9, k


@pytest.mark.gpu
def test_decoding_follows_the_sequence_form(cuda, lm):
    gen = torch.Generator().manual_seed(4)
    model = lm.RecurrentLM(64, 128, 2, torch.float32, seed=6)
    tokens, target, reset = lm.synthetic(64, 20, 3, gen)
    _, ctx = model.forward(tokens, target, reset)
    pools = [torch.full((5, 128), 9.0, device="cuda") for _ in range(2)]
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    for pool in pools:
        pool[slots.long()] = 0.0
    for t in range(20):
        logits = model.decode(tokens[t], pools, slots, reset=reset[t])
    for i in range(2):
        assert float((pools[i][slots.long()] - ctx["states"][i]).abs().max()) <= 1e-4
        assert torch.equal(pools[i][[1, 3]], torch.full((2, 128), 9.0, device="cuda"))
    s, y, _, _ = ctx["end"]
    assert float((logits - y[-1].float() @ model.c["head"].float().t()).abs().max()) <= 1e-3
    # a sequence in two calls, its states handed over
    _, a = model.forward(tokens[:8], target[:8], reset[:8])
    loss, b = model.forward(tokens[8:], target[8:], reset[8:], states=a["states"])
    whole, _ = model.forward(tokens, target, reset)
    assert float((loss - whole[8:]).abs().max()) <= 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_training_learns(cuda, lm, bits):
    """bf16: the loss falls well below the uniform guess (log 64 = 4.16) in 60 steps."""
    gen = torch.Generator().manual_seed(7)
    model = lm.RecurrentLM(64, 128, 1, torch.bfloat16, seed=8)
    opt = lm.Optimizer(model, bits=bits)
    first = last = None
    for _ in range(60):
        last = float(lm.train_step(model, opt, lm.synthetic(64, 64, 8, gen)))
        first = last if first is None else first
    assert first > 3.5 and last < 2.0, (first, last)
    assert cuda.last_error() == cuda.LR_OK


def test_synthetic_targets_follow_from_their_tokens(lm):
    """Every target that counts is what one of the two rules makes of its token, the
    last step's as well, after which a document may start (CPU)."""
    gen = torch.Generator().manual_seed(6)
    for T in (1, 7, 64, 129):
        tok, target, reset = lm.synthetic(509, T, 32, gen, device="cpu")
        live = target != lm.IGNORE
        follows = (target == (tok + 1) % 509) | (target == (2 * tok + 1) % 509)
        assert bool(follows[live].all())
        assert reset.shape == (T, 32) and bool(reset[0].all())
        assert not bool(live[:-1][reset[1:].bool()].any())
