"""The order of the sums of the language-model operators."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,d", [(torch.float32, 512), (torch.bfloat16, 1024)])
def test_embedding_gradient_does_not_depend_on_alignment(t, d):
    """Ids in segments of thousands: their sums are joined from parts, whose bounds
    must not move with the access width that the rows' alignment allows."""
    n, V = 50000, 2000
    g = torch.Generator(device="cuda")
    g.manual_seed(41)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    ids[torch.rand(n, generator=g, device="cuda") < 0.6] = 7
    flat = torch.randn(n * d + 1, generator=g, device="cuda").to(t)
    moved, rows = flat[1:].view(n, d), flat[1:].clone().view(n, d)
    assert moved.data_ptr() % 16 and rows.data_ptr() % 16 == 0
    got, ref = nr.embedding_backward(ids, moved, V), nr.embedding_backward(ids, rows, V)
    assert torch.equal(got, ref)
