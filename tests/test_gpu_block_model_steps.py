"""The example model's steps against its whole sequences, normwise.

Both ways round the same values, but P, the gate and the feed-forward come from products in
another order, so that a value next to a rounding's border falls to the other side.  bf16: at
most a dozen such values a block of 2^-8 / sqrt(12) = 1.1e-3 each, two blocks, either way:
sqrt(48) 1.1e-3 = 0.8% if every one differed.  fp32: 2^-24 / sqrt(12), sums of 64 to 256
products another 2^-22: below 1e-5.  A state, a gate or a branch that is left out is of
order 1."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,tol", [(torch.float32, 1e-5), (torch.bfloat16, 8e-3)])
@pytest.mark.parametrize("slots", [1, 5, 40])
def test_steps_follow_the_whole_sequence(slots, t, tol):
    from language_model import LanguageModel
    torch.backends.cuda.matmul.allow_tf32 = False
    model = LanguageModel(vocab=200, d=64, blocks=2, dtype=t, seed=3, cell="linear", mlp=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(slots)
    tokens = torch.randint(0, 200, (slots, 12), generator=g, device="cuda")
    u, _ = model.forward(tokens)
    whole = model.logit_scale * u.float() @ model.weights["embed"].float().T
    states = None
    for j in range(tokens.shape[1]):
        logits, states = model.step(tokens[:, j].contiguous(), states)
        assert float((logits - whole[:, j]).norm() / whole[:, j].norm()) <= tol, j
