"""GPU tests of the language-model operators at the ends of the types' ranges."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64


def test_vocab_loss_gradients_next_to_the_largest_value():
    """A dL/dloss next to fp32's largest value: entries of G whose nearest bf16 is an
    infinity still split into planes that add up to them.  x and W are so small that
    every logit is zero, p = 1 / V, and both gradients are far from overflow.

    p is off by 2^-19 relative (lse and its product with log2(e) rounded at 7 to 10,
    the exponential); the six plane products and their accumulation add 2^-16 of
    the magnitudes at most."""
    n, V, d = 40, 1000, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(21)
    x = torch.randn(n, d, generator=g, device="cuda") * 1e-30
    W = torch.randn(V, d, generator=g, device="cuda") * 1e-30
    t = torch.randint(0, V, (n,), generator=g, device="cuda")
    gl = torch.full((n,), torch.finfo(torch.float32).max, device="cuda")
    gl[1::2] *= -1
    loss, lse = nr.vocab_loss(x, W, t)
    gx, gW = nr.vocab_loss_backward(x, W, t, lse, gl)
    G = torch.full((n, V), 1 / V, dtype=F64, device="cuda")
    G[torch.arange(n, device="cuda"), t] -= 1
    assert float(G.abs().max()) * torch.finfo(torch.float32).max > 3.3962e38   # beyond bf16's last midpoint
    G *= gl.to(F64)[:, None]
    for got, ref, mag in ((gx, G @ W.to(F64), G.abs() @ W.to(F64).abs()), (gW, G.T @ x.to(F64), G.abs().T @ x.to(F64).abs())):
        assert bool(got.isfinite().all())
        assert bool(((got.to(F64) - ref).abs() <= 2.0 ** -15 * mag).all())


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_vocab_loss_gradients_of_an_infinite_or_nan_row(t):
    """A dL/dloss that is no number reaches its own row of gx, all of gW, and no
    other row of gx."""
    n, V, d = 40, 300, 72
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    x, W = (torch.randn(*s, d, generator=g, device="cuda").to(t) for s in ((n,), (V,)))
    at = torch.randint(0, V, (n,), generator=g, device="cuda")
    gl = torch.ones(n, device="cuda")
    lse = nr.vocab_loss(x, W, at)[1]
    good = nr.vocab_loss_backward(x, W, at, lse, gl)[0]
    for bad in (float("inf"), float("-inf"), float("nan")):
        gl[7] = bad
        gx, gW = nr.vocab_loss_backward(x, W, at, lse, gl)
        assert not bool(gx[7].isfinite().any()) and not bool(gW.isfinite().any())
        rest = torch.arange(n, device="cuda") != 7
        assert torch.equal(gx[rest], good[rest])
