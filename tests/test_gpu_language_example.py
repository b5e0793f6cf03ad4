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
