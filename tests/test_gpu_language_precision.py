"""What rounding G to bf16 costs the gradients of a bf16 vocabulary loss, measured by
what rounding the exact gradients once costs (the least that a bf16 result can be off).

Up to 64 rows G is held to 2^-16, which adds nothing that shows: 1.05.  Above, its
entries are rounded to 2^-8, as the results are; where those roundings are independent
of each other the two add up to sqrt(2) of one, held to 1.45.  They are not where all
rows' largest entries, (1 - p) dL/dloss, share a mantissa close above one: dL/dloss =
1/n for 15, 100, 250, 1000, 1500 rows here."""
import math

import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64


def inputs(n, V, d, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W = (torch.randn(V, d, generator=g, device="cuda") * (2 / math.sqrt(d))).bfloat16()
    t = ((float(V) ** torch.rand(n, generator=g, device="cuda", dtype=F64)).long().clamp_(1, V) - 1)
    lean = torch.rand(n, 1, generator=g, device="cuda") * 1.5         # some rows lean towards their target
    x = (torch.randn(n, d, generator=g, device="cuda") + lean * W[t].float()).bfloat16()
    return g, x, W, t


def over_rounding(x, W, t, gl, c=1.0):
    """The errors of gx and gW over those of the exact gradients rounded once."""
    lse = nr.vocab_loss(x, W, t, logit_scale=c)[1]
    got = nr.vocab_loss_backward(x, W, t, lse, gl, logit_scale=c)
    X, V = x.to(F64), W.to(F64)
    G = torch.softmax(c * X @ V.T, 1)
    G[torch.arange(t.numel(), device="cuda"), t] -= 1
    G *= c * gl[:, None].to(F64)
    return [float((o.to(F64) - r).norm() / (r.bfloat16().to(F64) - r).norm()) for o, r in zip(got, (G @ V, G.T @ X))]


@pytest.mark.parametrize("n", [1, 2, 4, 7, 15, 40, 64])
def test_few_rows(n):
    for seed in range(5):
        g, x, W, t = inputs(n, 3000, 128, 80 + seed)
        for gl, c in ((torch.full((n,), 1 / n, device="cuda"), 1.0), (torch.randn(n, generator=g, device="cuda"), 0.7)):
            over = over_rounding(x, W, t, gl, c)
            assert max(over) <= 1.05, (seed, c, over)


@pytest.mark.parametrize("n,V,d", [(65, 3000, 128), (100, 3000, 128), (250, 3000, 515), (1000, 5000, 64), (1500, 3000, 128),
                                   (4100, 9000, 256), (15000, 700, 128)])
def test_many_rows(n, V, d):
    g, x, W, t = inputs(n, V, d, 90)
    for gl, c in ((torch.full((n,), 1 / n, device="cuda"), 1.0), (torch.full((n,), -1.03, device="cuda"), 1.0),
                  (torch.randn(n, generator=g, device="cuda"), 0.7)):
        over = over_rounding(x, W, t, gl, c)
        print(n, ["%.2f" % o for o in over])
        assert max(over) <= 1.45, (c, over)


@pytest.mark.parametrize("n", [40, 300])
def test_a_first_row_of_any_weight(n):
    """The first kept row's dL/dloss sets nothing but a power of two: zero, tiny, huge."""
    g, x, W, t = inputs(n, 900, 96, 95)
    gl = torch.ones(n, device="cuda")
    for first in (0.0, 1e-40, 3e38, -1.99):
        gl[0] = first
        lse = nr.vocab_loss(x, W, t)[1]
        gx, gW = nr.vocab_loss_backward(x, W, t, lse, gl)
        rest = torch.arange(n, device="cuda") > 0
        alone = nr.vocab_loss_backward(x[rest], W, t[rest], lse[rest], gl[rest])
        a, b = gx[rest].to(F64), alone[0].to(F64)
        assert float((a - b).norm() / b.norm()) <= 2.0 ** -6
        if first == 0.0:
            assert bool((gx[0] == 0).all())
            assert float((gW.to(F64) - alone[1].to(F64)).norm() / alone[1].to(F64).norm()) <= 2.0 ** -6
    none = torch.full_like(t, -100)
    gx, gW = nr.vocab_loss_backward(x, W, none, lse, gl)
    assert bool((gx == 0).all()) and bool((gW == 0).all())


@pytest.mark.parametrize("n,V,d", [(1, 14045, 768), (2, 14045, 768), (3, 30000, 640)])
def test_fp32_gradient_of_a_few_rows(n, V, d):
    """A row of gx is one row of W and small terms after it.  The tensor cores drop up to
    2^-23 of the running sum, half of it on average, at each of an accumulator's steps
    of 16 products: 16 steps (256 elements) are 2^-20 of the whole."""
    for seed in range(4):
        g, x, W, t = inputs(n, V, d, 100 + seed)
        x, W = x.float() * 1.001, W.float() * 1.001
        gl = torch.full((n,), 1 / n, device="cuda")
        lse = nr.vocab_loss(x, W, t)[1]
        gx, _ = nr.vocab_loss_backward(x, W, t, lse, gl)
        G = torch.softmax(x.to(F64) @ W.to(F64).T, 1)
        G[torch.arange(n, device="cuda"), t] -= 1
        ref = G @ W.to(F64) * gl[:, None].to(F64)
        off = float((gx.to(F64) - ref).norm() / ref.norm())
        print(n, "%.1e" % off)
        assert off <= 2.0 ** -20
