"""The block operators and the fast-weight layer together, as examples/hybrid_model.py
runs them: training, gradients against torch's autograd of the same model in 64
bits, and decoding against prefilling the same tokens."""
from __future__ import annotations

import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
from hybrid_model import HybridModel, documents  # noqa: E402
from parity_check import rel_fro, report  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def plain_loss(params, blocks, fast, chunk, eta, d, tokens, targets, starts):
    """The model's loss in 64-bit torch operations (token by token, chunk by chunk)."""
    def norm(x, name):
        m = x.mean(-1, keepdim=True)
        v = ((x - m) ** 2).mean(-1, keepdim=True)
        return (x - m) / torch.sqrt(v + 1e-5) * params[name + ".gamma"] + params[name + ".beta"]

    e = params["embed"][tokens]
    h = e
    n, length = tokens.shape
    for i in range(blocks):
        gv = norm(h, f"{i}.mix") @ params[f"{i}.w_mix"].T
        f, v = torch.sigmoid(gv[..., :d]), gv[..., d:]
        s, rows = torch.zeros_like(v[:, 0]), []
        for t in range(length):
            keep = (starts[:, t] == 0)[:, None]
            s = f[:, t] * s * keep + (1 - f[:, t]) * v[:, t]
            rows.append(s)
        h = h + torch.stack(rows, 1) @ params[f"{i}.w_out"].T
        y = norm(h, f"{i}.mlp")
        z = torch.nn.functional.silu(y @ params[f"{i}.w_gate"].T) * (y @ params[f"{i}.w_up"].T)
        if i not in fast:
            h = h + z @ params[f"{i}.w_down"].T
            continue
        outs = []
        for b in range(n):
            w = params[f"{i}.w_down"].T
            for at in range(0, length, chunk):
                zc, ec = z[b, at:at + chunk], e[b, at:at + chunk]
                outs.append(zc @ w)
                pad = torch.cat([ec, torch.zeros(3, d, dtype=ec.dtype)])
                c = sum(params[f"{i}.conv_w"][:, j] * pad[j:j + ec.shape[0]] for j in range(4))
                w = w + eta * zc.T @ (c @ params[f"{i}.proj"].T)
        h = h + torch.cat(outs).view(n, length, d)
    logits = norm(h, "final") @ params["embed"].T
    return torch.nn.functional.cross_entropy(logits.flatten(0, 1), targets.flatten())


def test_gradients_against_autograd():
    """bf16 operators through 2 blocks against the 64-bit model with the same bf16 weights.
    Each gradient passes a few tens of bf16 roundings (1.7e-3 each in the mean square,
    adding in quadrature, amplified by the norms): 5e-2."""
    model = HybridModel(vocab=64, max_seq_len=192, eta=1e-2)
    tokens, targets, starts = documents(2, 192, 64, seed=3)
    loss, grads = model.loss_and_grads(tokens, targets, starts)
    p = {k: v.double().cpu().requires_grad_() for k, v in model.w.items()}
    for i in model.fast:   # the fast weight's start is fp32
        p[f"{i}.w_down"] = model.params[f"{i}.w_down"].double().cpu().requires_grad_()
    want = plain_loss(p, model.blocks, model.fast, model.chunk, model.eta, model.d, tokens.cpu(),
                      targets.cpu(), starts.cpu())
    want.backward()
    assert abs(loss.item() - want.item()) <= 2e-2 * want.item()
    assert set(grads) == set(p)
    for k in sorted(p):
        err = rel_fro(grads[k].double().cpu().numpy(), p[k].grad.numpy())
        report(f"[hybrid model] d {k}: rel_fro {err:.2e}")
        assert err <= 5e-2, (k, err)


def test_training_lowers_the_loss():
    model = HybridModel(vocab=64, max_seq_len=256)
    losses = [model.step(*documents(2, 256, 64, seed=k)) for k in range(12)]
    report(f"[hybrid model] loss {losses[0]:.3f} -> {losses[-1]:.3f}")
    assert losses[-1] < 0.8 * losses[0]


def test_decoding_equals_prefilling():
    """128 prompt tokens, then 100 token by token (the fast weight completes a chunk in
    between), against one prefill of the 256 tokens that start with them."""
    model = HybridModel(vocab=64, max_seq_len=256)
    tokens, _, _ = documents(2, 256, 64, seed=5)
    whole = model.prefill(tokens).float()
    first = model.prefill(tokens[:, :128]).float()
    assert rel_fro(first.cpu().numpy(), whole[:, :128].cpu().numpy()) <= 1e-2
    worst = 0.0
    for t in range(128, 228):
        got = model.decode(tokens[:, t]).float()
        worst = max(worst, rel_fro(got.cpu().numpy(), whole[:, t].cpu().numpy()))
    report(f"[hybrid model] decode against prefill: worst rel_fro {worst:.2e}")
    # the two differ by bf16 roundings in other places: those of one pass, 5e-2
    assert worst <= 5e-2
