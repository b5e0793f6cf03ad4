"""GPU parity of the gated feed-forward block against float64.

Tolerances, element by element.  A sum of K products is off by at most (K + 64) 2^-24
of the products' magnitudes (fp32 sums in any order; the tensor cores' drop up to
2^-23 of the running magnitude a step of 16, and fp32 factors are split to 2^-24);
the gate's exponential and reciprocal add 2^-20 of its value.  For bf16, m = silu(a) b
is rounded before the second product (2^-8), a and b as kept for the gradient, dL/da,
dL/db and the results likewise.  Each bound goes through the next product."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = [torch.float32, torch.bfloat16]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, t=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)


def inputs(n, d, f, t, seed=0):
    g = gen(seed)
    return (randn(g, n, d, t=t), randn(g, 2 * f, d, t=t, std=d ** -0.5), randn(g, d, f, t=t, std=f ** -0.5),
            randn(g, n, d, t=t))


def reference(x, W_in, W_out, g=None):
    """Results and bounds of their errors, in float64."""
    t = x.dtype
    u = 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24
    x, W_in, W_out = x.to(F64), W_in.to(F64), W_out.to(F64)
    n, d = x.shape
    f = W_out.shape[1]

    def s(k):
        return (k + 64) * 2.0 ** -24
    ab = x @ W_in.T
    eab = s(d) * (x.abs() @ W_in.abs().T)
    a, b, ea, eb = ab[:, :f], ab[:, f:], eab[:, :f], eab[:, f:]
    sig = torch.sigmoid(a)
    silu, dsilu = a * sig, sig * (1 + a * (1 - sig))
    m = silu * b
    # |silu'| <= 1.1, |silu''| <= 0.5
    em = 1.1 * ea * b.abs() + silu.abs() * eb + 1.1 * ea * eb + 2.0 ** -20 * m.abs()
    em = em + u * (m.abs() + em)
    y = m @ W_out.T
    ey = em @ W_out.abs().T + s(f) * (m.abs() @ W_out.abs().T)
    ey = ey + u * (y.abs() + ey)
    if g is None:
        return y, ey
    g = g.to(F64)
    ka, kb = ea + u * (a.abs() + ea), eb + u * (b.abs() + eb)      # as kept
    gm = g @ W_out
    egm = s(d) * (g.abs() @ W_out.abs())
    egm = egm + u * (gm.abs() + egm)
    ga, gb = gm * b * dsilu, gm * silu
    ega = egm * (b.abs() + kb) * 1.1 + gm.abs() * (kb * 1.1 + b.abs() * 0.5 * ka) + 2.0 ** -19 * gm.abs() * b.abs()
    egb = egm * (silu.abs() + 1.1 * ka) + gm.abs() * 1.1 * ka + 2.0 ** -20 * gb.abs()
    gab = torch.cat([ga, gb], 1)
    egab = torch.cat([ega, egb], 1)
    egab = egab + u * (gab.abs() + egab)
    gx = gab @ W_in
    egx = egab @ W_in.abs() + s(2 * f) * (gab.abs() @ W_in.abs())
    gWi = gab.T @ x
    eWi = egab.T @ x.abs() + s(n) * (gab.abs().T @ x.abs())
    gWo = g.T @ m
    eWo = g.abs().T @ em + s(n) * (g.abs().T @ m.abs())
    return y, ey, gx, egx + u * (gx.abs() + egx), gWi, eWi + u * (gWi.abs() + eWi), gWo, eWo + u * (gWo.abs() + eWo)


def check(got, ref, tol, what):
    got = got.to(F64)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - ref).abs().max()), bad.nonzero()[:4].tolist())


def check_norm(got, ref, t, what):
    """Normwise: roundings are spread as errors of either sign, so a chain of them leaves
    a few times one rounding's root mean square (2^-8 / sqrt(12) and 2^-24 sqrt(K))."""
    off = float((got.to(F64) - ref).norm() / ref.norm())
    assert off <= (2.0 ** -7.5 if t == torch.bfloat16 else 3e-6), (what, off)


SIZES = [(1, 8, 8), (1, 64, 128), (2, 40, 24), (3, 33, 7), (4, 1024, 512), (7, 250, 683), (16, 264, 300), (17, 64, 64),
         (64, 136, 264), (65, 512, 100), (128, 64, 128), (129, 72, 130), (255, 256, 256), (300, 130, 514), (513, 96, 1032),
         (1000, 64, 40)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d,f", SIZES)
def test_forward_and_backward(n, d, f, t):
    x, W_in, W_out, g = inputs(n, d, f, t, seed=n + d + f)
    y, ey, gx, egx, gWi, eWi, gWo, eWo = reference(x, W_in, W_out, g)
    got = nr.gated_mlp(x, W_in, W_out)
    check(got, y, ey, "y")
    got, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    check(got, y, ey, "y kept")
    r = nr.gated_mlp_backward(x, W_in, W_out, kept, g)
    check(r[0], gx, egx, "gx")
    check(r[1], gWi, eWi, "gW_in")
    check(r[2], gWo, eWo, "gW_out")
    again = nr.gated_mlp_backward(x, W_in, W_out, kept, g)
    assert all(torch.equal(p, q) for p, q in zip(r, again))
    assert torch.equal(got, nr.gated_mlp(x, W_in, W_out, keep=True)[0])


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d,f", [(3000, 250, 683), (2500, 512, 1024), (6, 512, 2000), (5000, 1024, 264)])
def test_accuracy(n, d, f, t):
    x, W_in, W_out, g = inputs(n, d, f, t, seed=1)
    y, _, gx, _, gWi, _, gWo, _ = reference(x, W_in, W_out, g)
    got, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    check_norm(got, y, t, "y")
    for p, q, what in zip(nr.gated_mlp_backward(x, W_in, W_out, kept, g), (gx, gWi, gWo), ("gx", "gW_in", "gW_out")):
        check_norm(p, q, t, what)


def test_gradients_against_differences():
    n, d, f = 5, 12, 20
    x, W_in, W_out, g = inputs(n, d, f, torch.float32, seed=2)
    _, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    got = nr.gated_mlp_backward(x, W_in, W_out, kept, g)

    def value(x, W_in, W_out):
        ab = x @ W_in.T
        return ((ab[:, :f] * torch.sigmoid(ab[:, :f]) * ab[:, f:]) @ W_out.T * g.to(F64)).sum()
    at = [x.to(F64), W_in.to(F64), W_out.to(F64)]
    for which in range(3):
        for i in range(0, at[which].numel(), max(1, at[which].numel() // 15)):
            pair = []
            for sign in (1, -1):
                moved = [v.clone() for v in at]
                moved[which].view(-1)[i] += sign * 1e-5
                pair.append(value(*moved))
            slope = float((pair[0] - pair[1]) / 2e-5)
            assert abs(float(got[which].view(-1)[i]) - slope) <= 2e-5 * (1 + abs(slope)), (which, i)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [3, 200])
def test_strides_alignment_shapes_and_outputs(n, t):
    d, f = 72, 136
    x, W_in, W_out, g = inputs(n, d, f, t, seed=5)
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    r = nr.gated_mlp_backward(x, W_in, W_out, kept, g)

    def shifted(v):                                      # the same values an element past alignment
        return torch.cat([v.reshape(-1)[:1], v.reshape(-1)])[1:].view(v.shape)
    out = shifted(torch.zeros_like(y))
    y2 = nr.gated_mlp(shifted(x), shifted(W_in), shifted(W_out), out=out)
    assert y2 is out
    ref, tol = reference(x, W_in, W_out)[:2]
    check(y2, ref, tol, "unaligned")
    y3, kept3 = nr.gated_mlp(shifted(x), shifted(W_in), shifted(W_out), keep=True)
    refs = reference(x, W_in, W_out, g)
    for got, ref, tol in zip(nr.gated_mlp_backward(shifted(x), shifted(W_in), shifted(W_out), kept3, shifted(g)), refs[2::2], refs[3::2]):
        check(got, ref, tol, "unaligned gradients")
    wide = torch.zeros(n, d + 3, dtype=t, device="cuda")
    wide[:, 1:d + 1] = x
    assert torch.equal(nr.gated_mlp(wide[:, 1:d + 1], W_in, W_out, keep=True)[0], y)
    assert torch.equal(nr.gated_mlp(x, W_in.t().contiguous().t(), W_out, keep=True)[0], y)
    assert torch.equal(nr.gated_mlp(x.view(1, n, d), W_in, W_out, keep=True)[0], y.view(1, n, d))


@pytest.mark.parametrize("t", TYPES)
def test_empty_and_refusals(t):
    x, W_in, W_out, g = inputs(4, 16, 24, t)
    y, kept = nr.gated_mlp(x[:0], W_in, W_out, keep=True)
    assert y.shape == (0, 16)
    gx, gWi, gWo = nr.gated_mlp_backward(x[:0], W_in, W_out, kept, g[:0])
    assert gx.shape == (0, 16) and not bool(gWi.any()) and not bool(gWo.any())
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    for call in (lambda: nr.gated_mlp(x.cpu(), W_in, W_out), lambda: nr.gated_mlp(x, W_in[:47], W_out),
                 lambda: nr.gated_mlp(x, W_in, W_out.t()), lambda: nr.gated_mlp(x[:, :8], W_in, W_out),
                 lambda: nr.gated_mlp(x, W_in, W_out, out=torch.empty(3, 16, dtype=t, device="cuda")),
                 lambda: nr.gated_mlp(x, W_in, W_out, workspace=torch.empty(1 << 22, dtype=torch.uint8)),
                 lambda: nr.gated_mlp_backward(x, W_in, W_out, kept[:-1], g),
                 lambda: nr.gated_mlp_backward(x, W_in, W_out, kept, g[:3]),
                 lambda: nr.gated_mlp_backward(x, W_in, W_out, kept.cpu(), g),
                 lambda: nr.gated_mlp_backward(x[:3], W_in, W_out, kept, g[:3])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nr.gated_mlp(x.double(), W_in.double(), W_out.double())
    with pytest.raises(TypeError):
        nr.gated_mlp(x, W_in.double(), W_out)


def test_rows_do_not_mix():
    """A row that holds NaN or infinities reaches no other row of y or gx."""
    n, d, f = 300, 64, 128
    for t in TYPES:
        x, W_in, W_out, g = inputs(n, d, f, t, seed=8)
        y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
        gx = nr.gated_mlp_backward(x, W_in, W_out, kept, g)[0]
        x2 = x.clone()
        x2[131], x2[7] = float("nan"), float("inf")
        y2, kept2 = nr.gated_mlp(x2, W_in, W_out, keep=True)
        gx2 = nr.gated_mlp_backward(x2, W_in, W_out, kept2, g)[0]
        live = torch.ones(n, dtype=torch.bool, device="cuda")
        live[[131, 7]] = False
        assert torch.equal(y[live], y2[live]) and torch.equal(gx[live], gx2[live])
        assert bool(y2[131].isnan().all()) and not bool(y2[7].isfinite().any())


@pytest.mark.parametrize("t", TYPES)
def test_large_and_small_preactivations(t):
    """Gates far from zero: silu(a) is a or 0 to the last bit, and nothing is infinite or NaN."""
    x, W_in, W_out, g = inputs(40, 64, 128, t, seed=9)
    for scale in (40.0, 3000.0, 1e-6):
        W = W_in.clone()
        W[:128] *= scale
        y, kept = nr.gated_mlp(x, W, W_out, keep=True)
        refs = reference(x, W, W_out, g)
        check(y, refs[0], refs[1], ("y", scale))
        for got, ref, tol in zip(nr.gated_mlp_backward(x, W, W_out, kept, g), refs[2::2], refs[3::2]):
            check(got, ref, tol, scale)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [5, 300])
def test_streams_and_capture(n, t):
    d, f = 128, 264
    x, W_in, W_out, g = inputs(n, d, f, t, seed=10)
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    r = nr.gated_mlp_backward(x, W_in, W_out, kept, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, kept1 = nr.gated_mlp(x, W_in, W_out, keep=True)
        r1 = nr.gated_mlp_backward(x, W_in, W_out, kept1, g)
    y2, kept2 = nr.gated_mlp(x, W_in, W_out, keep=True)           # at the same time, on this stream
    r2 = nr.gated_mlp_backward(x, W_in, W_out, kept2, g)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in ((y1, r1), (y2, r2)):
        assert torch.equal(a, y) and all(torch.equal(p, q) for p, q in zip(b, r))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, keptg = nr.gated_mlp(x, W_in, W_out, keep=True)
        rg = nr.gated_mlp_backward(x, W_in, W_out, keptg, g)
    x.copy_(inputs(n, d, f, t, seed=11)[0])
    graph.replay()
    y3, kept3 = nr.gated_mlp(x, W_in, W_out, keep=True)
    r3 = nr.gated_mlp_backward(x, W_in, W_out, kept3, g)
    assert torch.equal(yg, y3) and all(torch.equal(p, q) for p, q in zip(rg, r3))


def test_offsets_beyond_32_bits():
    """The last rows of more than 2^32 kept values; with g zero before them the gradients
    of the weights are theirs too."""
    n, d, f, k = (1 << 20) + 77, 8, 4104, 300
    assert n * f > 1 << 32
    x, W_in, W_out, g = inputs(n, d, f, torch.bfloat16, 5)
    g[:-k] = 0
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    gx, gWi, gWo = nr.gated_mlp_backward(x, W_in, W_out, kept, g)
    ry, ey, rx, ex, ri, ei, ro, eo = reference(x[-k:], W_in, W_out, g[-k:])
    check(y[-k:], ry, ey, "y")
    check(gx[-k:], rx, ex, "gx")
    check(gWi, ri, ei, "gW_in")
    check(gWo, ro, eo, "gW_out")
    assert not bool(gx[:-k].any())
