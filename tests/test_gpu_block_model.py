"""The block's operators run together, as the example model does: every weight's gradient
against float64 differentiation of the same model written out with elementary operations,
a step at a time against the whole sequence, and a packed prefill that goes on in steps.

Tolerances: fp32 operators leave under 1e-5 of their results' size each, the norms and
the way through the blocks and back multiply that by less than a hundred; a missing term
is of order 1."""
import os
import sys

import pytest
import torch

import nonlinear_rnn_gb300 as nr

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

EPS = 1e-6


def norm(v):
    return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt()


def reference_loss(w, tokens, targets, model, ignore, keeps):
    x = w["embed"][tokens] * model.embed_scale
    u = norm(x) * w["0.w_pre"]
    for b in range(model.blocks):
        pa, pi, v = (u @ w[f"{b}.W_x"].T).chunk(3, -1)
        log_rate, b_a, b_i = w[f"{b}.cell"]
        a = torch.exp(-log_rate.exp() * torch.sigmoid(pa + b_a))
        new = torch.sqrt(1 - a * a) * torch.sigmoid(pi + b_i) * v
        h, states = torch.zeros_like(v[:, 0]), []
        for t in range(tokens.shape[1]):
            h = a[:, t] * h + new[:, t]
            states.append(h)
        gate = u @ w[f"{b}.W_gate"].T
        x = x + w[f"{b}.scale"] * norm(torch.stack(states, 1)) * w[f"{b}.w_post"] * gate * torch.sigmoid(gate)
        last = "w_out" if b + 1 == model.blocks else f"{b + 1}.w_pre"
        if model.mlp:
            ab = norm(x) * w[f"{b}.w_mlp"] @ w[f"{b}.W_in"].T
            p, q = ab.chunk(2, -1)
            x = x + keeps[b] * ((p * torch.sigmoid(p) * q) @ w[f"{b}.W_out"].T) / (1 - model.p)
        u = norm(x) * w[last]
    logits = model.logit_scale * u @ w["embed"].T
    live = targets != ignore
    picked = torch.log_softmax(logits, -1).gather(-1, torch.where(live, targets, 0)[..., None])[..., 0]
    return -(picked * live).sum() / live.sum()


@pytest.mark.parametrize("blocks,d,vocab,mlp,p", [(2, 24, 61, 3, 0.25), (3, 40, 300, 0, 0.0), (1, 64, 90, 2, 0.5)])
def test_every_weight_of_the_model(blocks, d, vocab, mlp, p):
    from language_model import IGNORE, LanguageModel
    torch.backends.cuda.matmul.allow_tf32 = False
    model = LanguageModel(vocab=vocab, d=d, blocks=blocks, dtype=torch.float32, seed=5, cell="linear", mlp=mlp, p=p)
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    for name, v in model.weights.items():      # norm weights and scales that differ by column
        if v.dim() == 1:
            v += 0.3 * torch.randn(v.shape, generator=g, device="cuda")
    tokens = torch.randint(0, vocab, (3, 70), generator=g, device="cuda")
    targets = torch.randint(0, vocab, (3, 70), generator=g, device="cuda")
    targets[0, :7] = IGNORE
    loss, grads = model.gradients(tokens, targets, step=9)
    assert torch.equal(loss, model.loss(tokens, targets, step=9))
    keeps = [(nr.dropout(torch.ones(3, 70, d, device="cuda"), p, 9, offset=b) > 0).cpu().double() for b in range(blocks)]
    w = {k: v.cpu().double().requires_grad_(True) for k, v in model.weights.items()}
    ref = reference_loss(w, tokens.cpu(), targets.cpu(), model, IGNORE, keeps)
    assert abs(float(loss) - float(ref.detach())) <= 1e-4
    ref_grads = dict(zip(w, torch.autograd.grad(ref, list(w.values()))))
    assert set(grads) == set(ref_grads)
    for name, r in ref_grads.items():
        off = float((grads[name].cpu().double() - r).norm() / r.norm())
        assert off <= 1e-3, (name, off)


@pytest.mark.parametrize("t,tol", [(torch.float32, 1e-3), (torch.bfloat16, 0.25)])
def test_steps_follow_the_whole_sequence(t, tol):
    """Logits of order 1 to 5.  bf16 roundings of two blocks' activations (2^-8 each, a dozen
    of them) leave up to a few hundredths of the logits' size."""
    from language_model import LanguageModel
    model = LanguageModel(vocab=200, d=64, blocks=2, dtype=t, seed=3, cell="linear", mlp=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    tokens = torch.randint(0, 200, (5, 12), generator=g, device="cuda")
    u, _ = model.forward(tokens)
    whole = u.float() @ model.weights["embed"].float().T
    states = None
    for j in range(tokens.shape[1]):
        logits, states = model.step(tokens[:, j].contiguous(), states)
        assert float((logits - whole[:, j]).abs().max()) <= tol
    assert all(s.dtype == torch.float32 for s in states)


def test_a_packed_prefill_goes_on_in_steps():
    """Prompts of uneven length (one empty) prefilled as one pack, their last states taken on
    step by step, against each sequence alone."""
    lengths, d, more = [70, 0, 5, 130], 64, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    params = torch.stack([torch.rand(d, generator=g, device="cuda") + 0.01, torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    parts = [torch.randn(1, n + more, 3 * d, generator=g, device="cuda") for n in lengths]
    pack = torch.cat([p[:, :n] for p, n in zip(parts, lengths)], 1)
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    _, states = nr.linear_recurrence(pack, params, cu_seqlens=cu)
    for j in range(more):
        step = torch.cat([p[:, n + j] for p, n in zip(parts, lengths)])
        h, states = nr.linear_recurrence_step(params, states, step)
        for k, (p, n) in enumerate(zip(parts, lengths)):
            alone = nr.linear_recurrence(p[:, :n + j + 1], params)[0][0, -1]
            assert float((alone - h[k]).abs().max()) <= 1e-5      # states of order 1, fp32 roundings


def test_training_runs():
    from language_model import train
    losses = train(8, vocab=100, d=64, blocks=2, B=4, T=48, cell="linear", mlp=2, p=0.1)
    assert len(losses) == 8 and all(v == v and abs(v) < 100 for v in losses)


def test_readme_usage():
    """The README's example of the block's operators at a small size."""
    d, f = 64, 256
    x = torch.randn(2, 100, d, device="cuda", dtype=torch.bfloat16)
    W_x = torch.randn(3 * d, d, device="cuda", dtype=torch.bfloat16) / 8
    rate = torch.rand(d, device="cuda") * 0.5 + 0.01
    rec = torch.stack([rate, torch.zeros_like(rate), torch.zeros_like(rate)])
    P = nr.input_projection(x, W_x)
    H, last = nr.linear_recurrence(P, rec)
    g = nr.linear_recurrence_backward(P, rec, H, torch.ones_like(H))
    h, last2 = nr.linear_recurrence_step(rec, last, P[:, -1])
    W_in = torch.randn(2 * f, d, device="cuda", dtype=torch.bfloat16) / 8
    W_out = torch.randn(d, f, device="cuda", dtype=torch.bfloat16) / 16
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    z = nr.dropout(y, 0.1, seed=1, offset=0, residual=x)
    gy = nr.dropout(torch.ones_like(z), 0.1, seed=1, offset=0)
    grads = nr.gated_mlp_backward(x, W_in, W_out, kept, gy)
    assert g.gP.shape == P.shape and h.shape == (2, d) and z.shape == x.shape
    assert torch.equal(gy == 0, (z == x) & (gy == 0))       # what is dropped leaves the residual
    assert all(bool(t.isfinite().all()) for t in (H, last, last2, z, *g[:2], *grads))
