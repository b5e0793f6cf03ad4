"""Refusals of the language-model operators beyond shapes and types."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


def test_block_norm_without_h_has_nothing_for_out():
    x = torch.randn(4, 16, device="cuda")
    with pytest.raises(ValueError):
        nr.block_norm(x, out=torch.empty_like(x))
    first, u = nr.block_norm(x, out=x)
    assert first is x and torch.equal(u, nr.block_norm(x)[1])
