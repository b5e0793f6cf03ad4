"""The example model: its gradients against differences of its loss, and training."""
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_of_the_whole_model_against_differences():
    """Central differences of the fp32 loss along a random direction of every
    weight.  The loss is a mean of order 5: its rounding (about 2^-20) over the
    step and the third derivative's step^2 bound the error; K = 8 Newton
    iterations put H at the recurrence's fixed point, where the backward holds."""
    from language_model import IGNORE, LanguageModel
    model = LanguageModel(vocab=61, d=24, blocks=2, dtype=torch.float32, K=8, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tokens = torch.randint(0, 61, (3, 40), generator=g, device="cuda")
    targets = torch.randint(0, 61, (3, 40), generator=g, device="cuda")
    targets[0, :7] = IGNORE
    torch.backends.cuda.matmul.allow_tf32 = False
    loss, grads = model.gradients(tokens, targets)
    assert abs(float(loss) - float(model.loss(tokens, targets))) < 1e-5
    assert set(grads) == set(model.weights)
    step = 1e-2
    for name, grad in grads.items():
        to = torch.randn(grad.shape, generator=g, device="cuda")
        to /= to.norm()
        base = model.weights[name]
        values = []
        for s in (step, -step):
            model.weights[name] = base + s * to
            values.append(float(model.loss(tokens, targets)))
        model.weights[name] = base
        num = (values[0] - values[1]) / (2 * step)
        assert abs(num - float((grad * to).sum())) <= 20 * step ** 2 + 16 * 2.0 ** -20 / step, name


def test_training_lowers_the_loss():
    from language_model import train
    losses = train(60, vocab=300, d=128, blocks=2, B=8, T=64)
    assert all(math.isfinite(v) for v in losses)
    assert losses[0] > 0.9 * math.log(300)
    assert sum(losses[-5:]) / 5 < 0.6 * losses[0]


def test_readme_usage_of_the_language_operators():
    """The README's second example at a small size."""
    import nonlinear_rnn_gb300 as nr
    d, V = 64, 200
    W_x = (torch.randn(3 * d, d, device="cuda") / d ** 0.5).to(torch.bfloat16)
    params = torch.rand(6, d) * 2 - 1
    E = torch.randn(V, d, device="cuda", dtype=torch.bfloat16) / d ** 0.5
    tokens = torch.randint(0, V, (2, 48), device="cuda")
    targets = tokens.roll(-1, 1)
    x0 = nr.embedding(tokens, E, scale=8.0)
    _, u = nr.block_norm(x0)
    H, _ = nr.newton_forward(nr.input_projection(u, W_x), params, check=False)
    x1, v = nr.block_norm(x0, h=H)
    loss, lse = nr.vocab_loss(v, E, targets)
    gv, gE = nr.vocab_loss_backward(v, E, targets, lse, torch.full_like(loss, 1 / loss.numel()))
    g = nr.block_norm_backward(x1, h=H, g_u=gv)
    before = gE.clone()
    nr.embedding_backward(tokens, g.gx, V, scale=8.0, out=gE, accumulate=True)
    assert loss.shape == (2, 48) and gv.shape == v.shape and gE.shape == E.shape
    assert all(bool(t.isfinite().all()) for t in (loss, gv, gE, g.gx, g.gh))
    assert not torch.equal(before, gE)
