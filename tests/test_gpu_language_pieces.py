"""The vocabulary loss's backward over more than one piece of the vocabulary, in either
type and at widths that no 16-byte row fits, all of gx and gW against float64.

fp32: logits of a few units over d <= 67 are off by some 2^-21, lse by its rounding at
8 to 14 (2^-21), the products by 2^-22: 2^-19 of the whole.  bf16: G's rounding and the
result's, 2^-8 each, held to 2^-7 together.  A piece left out or added twice is of the
order of the pieces' number off."""
import math

import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64


@pytest.mark.parametrize("n,V,d,t", [
    (90000, 4500, 67, torch.float32),      # three pieces of 2048 columns at most, gx in elements
    (90000, 7000, 67, torch.bfloat16),     # two
    (70000, 9000, 250, torch.bfloat16),
    (300, 400000, 20, torch.float32),      # two, of few row tiles: tiles of gx are cut
    (6, 750000, 36, torch.float32),        # two, of rows on the fp32 cores
    (6, 705000, 33, torch.float32),
])
def test_backward_in_pieces(n, V, d, t):
    g = torch.Generator(device="cuda")
    g.manual_seed(61)
    x = torch.randn(n, d, generator=g, device="cuda").to(t)
    W = (torch.randn(V, d, generator=g, device="cuda") * (2 / math.sqrt(d))).to(t)
    target = torch.randint(0, V, (n,), generator=g, device="cuda")
    target[1::5] = V - 1 - target[1::5] % 50            # the last piece's own
    target[torch.rand(n, generator=g, device="cuda") < 0.1] = -100
    target[0] = 3
    gl = torch.randn(n, generator=g, device="cuda")
    planes = 3 if t == torch.float32 else 1
    assert -(-n // 256) * 256 * V * 2 * planes > 1 << 30   # G does not fit one piece
    loss, lse = nr.vocab_loss(x, W, target)
    gx, gW = nr.vocab_loss_backward(x, W, target, lse, gl)
    W64, gW_ref = W.to(F64), torch.zeros(V, d, dtype=F64, device="cuda")
    gx_ref = torch.zeros(n, d, dtype=F64, device="cuda")
    step = max(1, 50_000_000 // V)
    for i in range(0, n, step):
        at = target[i:i + step]
        live = torch.nonzero(at != -100)[:, 0]
        X = x[i:i + step][live].to(F64)
        z = X @ W64.T
        G = torch.softmax(z, 1)
        G[torch.arange(live.numel(), device="cuda"), at[live]] -= 1
        G *= gl[i:i + step][live, None].to(F64)
        gx_ref[i + live] = G @ W64
        gW_ref += G.T @ X
    tol = 2.0 ** -19 if t == torch.float32 else 2.0 ** -7
    for got, ref in ((gx, gx_ref), (gW, gW_ref)):
        off = float((got.to(F64) - ref).norm() / ref.norm())
        print(n, V, d, "%.1e" % off)
        assert off <= tol
    assert bool((gx[target == -100] == 0).all())
    again = nr.vocab_loss_backward(x, W, target, lse, gl)
    assert torch.equal(gx, again[0]) and torch.equal(gW, again[1])
