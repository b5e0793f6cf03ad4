"""The fp32 backward's probability of a class that has it all is one, whatever the logits' size.

x_i is a multiple of the row of W of its class, 48 its logit, beside which the others
vanish (e^-20): lse is that logit.  A column of W that only this class's row holds, against
zeros in x, gives p dL/dloss in gx as one product.  lse of [32, 64) is rounded by at most
2^-19, which p takes in full; the exponential adds 2^-22, the changes of base 2^-22."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.mark.parametrize("n,V,d", [(4, 900, 128), (16, 3000, 129), (16, 2000, 512), (300, 3000, 256), (600, 5000, 515)])
def test_a_certain_class_has_probability_one(n, V, d):
    g = torch.Generator(device="cuda")
    g.manual_seed(111)
    R = min(n, 48)                               # rows that are looked at, a column each
    W = torch.randn(V, d, generator=g, device="cuda")
    W[:, d - R:] = 0
    own = torch.randperm(V - 1, generator=g, device="cuda")[:n]
    # logits from 40 to 56: roundings of every kind
    at = 40 + 16 * torch.rand(n, 1, generator=g, device="cuda", dtype=F64)
    x = (W[own].to(F64) * at / W[own].to(F64).square().sum(1, keepdim=True)).float()
    W[own[:R], torch.arange(d - R, d, device="cuda")] = 1
    lse = nr.vocab_loss(x, W, torch.full_like(own, V - 1))[1]
    assert bool(((lse - at[:, 0]).abs() < 1e-3).all())
    gx, _ = nr.vocab_loss_backward(x, W, torch.full_like(own, V - 1), lse, torch.ones(n, device="cuda"))
    p = gx[torch.arange(R, device="cuda"), torch.arange(d - R, d, device="cuda")].to(F64)
    off = float((p - 1).abs().max())
    print(n, V, d, "%.1e" % off)
    assert off <= 2.0 ** -19 + 2.0 ** -21
