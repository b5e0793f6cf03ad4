"""The example model's gradients, weight by weight, against float64 differentiation of
the same model written out with elementary operations and a sequential recurrence.

Tolerance: the recurrent layer's states are within 2e-5 of the exact ones (its own
tests' bound), which the norm around it, of states of order 0.1 and above, turns into
2e-4 of a block's output; two blocks and the way back through both leave less than
2e-3 of a gradient.  Zeros, or a gradient that lacks one of its terms, are of order 1
off in the same measure."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

EPS = 1e-6


def norm(v):
    return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()


def reference_loss(w, tokens, targets, blocks, embed_scale, logit_scale, ignore):
    x = w["embed"][tokens] * embed_scale
    u = norm(x) * w["0.w_pre"]
    for b in range(blocks):
        pz, pr, pc = (u @ w[f"{b}.W_x"].T).chunk(3, -1)
        az, ar, ac, bz, br, bc = w[f"{b}.cell"]
        h, states = torch.zeros_like(pz[:, 0]), []
        for t in range(tokens.shape[1]):
            z = torch.sigmoid(pz[:, t] + az * h + bz)
            r = torch.sigmoid(pr[:, t] + ar * h + br)
            c = torch.tanh(pc[:, t] + ac * (r * h) + bc)
            h = (1 - z) * h + z * c
            states.append(h)
        gate = u @ w[f"{b}.W_gate"].T
        y = norm(torch.stack(states, 1)) * w[f"{b}.w_post"] * gate * torch.sigmoid(gate)
        x = x + w[f"{b}.scale"] * y
        u = norm(x) * w["w_out" if b + 1 == blocks else f"{b + 1}.w_pre"]
    logits = logit_scale * u @ w["embed"].T
    live = targets != ignore
    picked = torch.log_softmax(logits, -1).gather(-1, torch.where(live, targets, 0)[..., None])[..., 0]
    return -(picked * live).sum() / live.sum()


@pytest.mark.parametrize("blocks,d,vocab", [(2, 24, 61), (3, 40, 300)])
def test_every_weight_of_the_model(blocks, d, vocab):
    from language_model import IGNORE, LanguageModel
    torch.backends.cuda.matmul.allow_tf32 = False
    model = LanguageModel(vocab=vocab, d=d, blocks=blocks, dtype=torch.float32, K=8, seed=5)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for name, v in model.weights.items():      # norm weights and scales that differ by column
        if v.dim() == 1:
            v += 0.3 * torch.randn(v.shape, generator=g, device="cuda")
    tokens = torch.randint(0, vocab, (3, 40), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (3, 40), generator=g, device="cuda")
    targets[0, :7] = IGNORE
    loss, grads = model.gradients(tokens, targets)
    w = {k: v.cpu().double().requires_grad_(True) for k, v in model.weights.items()}
    ref = reference_loss(w, tokens.cpu(), targets.cpu(), blocks, model.embed_scale, model.logit_scale, IGNORE)
    assert abs(float(loss) - float(ref.detach())) <= 2e-4
    ref_grads = dict(zip(w, torch.autograd.grad(ref, list(w.values()))))
    assert set(grads) == set(ref_grads)
    for name, r in ref_grads.items():
        off = float((grads[name].cpu().double() - r).norm() / r.norm())
        print(name, "%.1e" % off)
        assert off <= 2e-3, (name, off)
