"""How exact the vocabulary loss is, as a whole: errors normwise against float64, so
that a bound does not grow with the vocabulary.

fp32: the errors of lse, gx and gW are at most three times those of the same formulas
in fp32 torch products (no TF32) on the same inputs.  Three sources stand in the
kernels where fp32 products have one: the plane products that are left out (2^-24 of
a product), the accumulation on the tensor cores, and the exponential and base-2
steps; each is of the size of fp32's own rounding.  lse has 2^-23 more for its two
changes of base.  test_the_bounds_tell_lesser_products_apart shows on the CPU that
zeros, bf16 products and products of two planes each lie outside.

bf16: G and the results are rounded to bf16, each by at most 2^-8 of an entry (8
significant bits); the two are independent, so 2^-8 sqrt(2), held to 2^-7; a row of a
result by itself to 2^-6.  The tensor cores add one step of 16 products after another,
each at most 2^-23 of the running sum off."""
import math

import pytest
import torch

import nonlinear_rnn_gb300 as nr

F64 = torch.float64
FP32_FACTOR, LSE_MORE = 3.0, 2.0 ** -23
BF16_WHOLE, BF16_ROW = 2.0 ** -7, 2.0 ** -6


def inputs(n, V, d, t, device, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    x = torch.randn(n, d, generator=g, device=device).to(t)
    W = (torch.randn(V, d, generator=g, device=device) * (2 / math.sqrt(d))).to(t)
    return x, W, torch.randint(0, V, (n,), generator=g, device=device), torch.randn(n, generator=g, device=device)


def formulas(x, W, t, gl, c, times=torch.matmul):
    """lse, gx, gW in the inputs' type, products by times(A, B) = A B."""
    z = c * times(x, W.T)
    lse = torch.logsumexp(z, 1)
    G = torch.exp(z - lse[:, None])
    G[torch.arange(t.numel(), device=t.device), t] -= 1
    G *= (gl.to(G.dtype) * c)[:, None]
    return lse, times(G, W), times(G.T, x)


def whole(got, ref):
    return float((got.to(F64) - ref).norm() / ref.norm())


def worst_row(got, ref):
    return float(((got.to(F64) - ref).norm(dim=1) / ref.norm(dim=1)).max())


def fp32_bounds(x, W, t, gl, c, ref):
    assert not torch.backends.cuda.matmul.allow_tf32
    plain = [whole(a, b) for a, b in zip(formulas(x, W, t, gl, c), ref)]
    return FP32_FACTOR * plain[0] + LSE_MORE, FP32_FACTOR * plain[1], FP32_FACTOR * plain[2]


def exact(x, W, t, gl, c):
    return formulas(x.to(F64), W.to(F64), t, gl, c)


def planes(v):
    out = []
    for _ in range(3):
        out.append(v.bfloat16().float())
        v = v - out[-1]
    return out


def by_planes(pairs):
    def times(A, B):
        a, b = planes(A), planes(B)
        return sum(a[i].to(F64) @ b[j].to(F64) for i, j in pairs).float()
    return times


SIX = ((2, 0), (1, 1), (0, 2), (1, 0), (0, 1), (0, 0))


@pytest.mark.parametrize("n,V,d", [(33, 2000, 96), (300, 5000, 515)])
def test_the_bounds_tell_lesser_products_apart(n, V, d):
    for c in (1.0, 8.0):
        args = (*inputs(n, V, d, torch.float32, "cpu", 51), c)
        ref = exact(*args)
        bounds = fp32_bounds(*args, ref)
        six = formulas(*args, times=by_planes(SIX))
        assert all(whole(o, r) <= b for o, r, b in zip(six, ref, bounds))
        for pairs in (((0, 0),), ((1, 0), (0, 1), (0, 0))):
            less = [whole(o, r) for o, r in zip(formulas(*args, times=by_planes(pairs)), ref)]
            assert less[1] > bounds[1] and less[2] > bounds[2]
            assert c == 1.0 or less[0] > bounds[0]
        assert whole(torch.zeros_like(ref[1]), ref[1]) > max(bounds[1], BF16_WHOLE)
        assert whole(torch.zeros_like(ref[2]), ref[2]) > max(bounds[2], BF16_WHOLE)


# rows of the fp32-core form (5, 16) and above, tiles of every orientation cut or whole
SIZES = [(5, 1000, 65), (16, 3000, 512), (33, 2000, 96), (300, 5000, 515), (513, 3001, 1024), (700, 33000, 96),
         (2100, 700, 250)]


@pytest.mark.gpu
@pytest.mark.parametrize("c", [1.0, 8.0])
@pytest.mark.parametrize("n,V,d", SIZES)
def test_fp32_loss_is_as_exact_as_fp32_products(n, V, d, c):
    x, W, t, gl = inputs(n, V, d, torch.float32, "cuda", 52)
    ref = exact(x, W, t, gl, c)
    lse = nr.vocab_loss(x, W, t, logit_scale=c)[1]
    got = (lse, *nr.vocab_loss_backward(x, W, t, lse, gl, logit_scale=c))
    errors, bounds = [whole(o, r) for o, r in zip(got, ref)], fp32_bounds(x, W, t, gl, c, ref)
    print(n, V, d, c, ["%.2g of %.2g" % p for p in zip(errors, bounds)])
    assert all(e <= b for e, b in zip(errors, bounds)), (errors, bounds)


@pytest.mark.gpu
@pytest.mark.parametrize("n,V,d", SIZES + [(8, 300, 16384)])
def test_bf16_loss_is_off_by_its_roundings(n, V, d):
    x, W, t, gl = inputs(n, V, d, torch.bfloat16, "cuda", 53)
    ref = exact(x, W, t, gl, 1.0)
    lse = nr.vocab_loss(x, W, t)[1]
    most = (x.to(F64) @ W.to(F64).T).abs().max(1).values
    off = (lse.to(F64) - ref[0]).abs()
    print(n, V, d, "lse off by %.2g of %.2g" % (float(off.max()), float(most.max())))
    # a logit's sum passes d / 16 steps; lse and the exponentials are rounded at its own size
    assert bool((off <= 2.0 ** -23 * (d / 16 + 8) * most + 2.0 ** -21 * (1 + ref[0].abs())).all())
    gx, gW = nr.vocab_loss_backward(x, W, t, lse, gl)
    for got, r in ((gx, ref[1]), (gW, ref[2])):
        assert whole(got, r) <= BF16_WHOLE and worst_row(got, r) <= BF16_ROW, (whole(got, r), worst_row(got, r))
