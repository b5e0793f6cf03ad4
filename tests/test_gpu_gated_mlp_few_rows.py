"""The feed-forward block of a decode step's rows: widths and tensors of which only some rows
are 16-byte aligned, and fp32 widths on both sides of what fits in shared memory."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr
from test_gpu_gated_mlp import TYPES, check, inputs, reference

pytestmark = pytest.mark.gpu


def shifted(v):
    """The same values an element past alignment."""
    return torch.cat([v.reshape(-1)[:1], v.reshape(-1)])[1:].view(v.shape)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("d,f", [(72, 131), (33, 136), (264, 515), (517, 264), (1024, 24), (8, 1000), (1, 1)])
@pytest.mark.parametrize("n", [1, 2, 4, 5, 8, 9, 16])
def test_widths(n, d, f, t):
    x, W_in, W_out, _ = inputs(n, d, f, t, seed=n + d)
    ref, tol = reference(x, W_in, W_out)
    check(nr.gated_mlp(x, W_in, W_out), ref, tol, "y")


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("which", range(1, 8))
@pytest.mark.parametrize("n", [1, 3, 8, 13])
def test_one_or_more_tensors_past_alignment(n, which, t):
    x, W_in, W_out, _ = inputs(n, 136, 264, t, seed=n)
    ref, tol = reference(x, W_in, W_out)
    x, W_in, W_out = (shifted(v) if which >> i & 1 else v for i, v in enumerate((x, W_in, W_out)))
    check(nr.gated_mlp(x, W_in, W_out), ref, tol, "y")


@pytest.mark.parametrize("n,d", [(8, 2817), (8, 2818), (8, 2824), (64, 2816), (64, 2824), (4, 5888), (4, 5896), (2, 5889), (2, 5890), (1, 24320),
                                 (1, 24328)])
def test_fp32_widths_beside_what_fits(n, d):
    f = 72
    x, W_in, W_out, _ = inputs(n, d, f, torch.float32, seed=d)
    ref, tol = reference(x, W_in, W_out)
    check(nr.gated_mlp(x, W_in, W_out), ref, tol, "y")


@pytest.mark.parametrize("n", [1, 8, 16, 17, 64])
def test_what_differs_by_the_rows_beside(n):
    """A bf16 row's y is rounded once in a call of at most 16 rows, and m before it in a longer
    one: within 1.5 roundings normwise (sqrt(2) and chance; one row: 256 results)."""
    x, W_in, W_out, _ = inputs(128, 256, 512, torch.bfloat16, seed=3)
    exact = reference(x[:n], W_in, W_out)[0]
    once = float((exact.to(torch.bfloat16).double() - exact).norm())
    for y, of in ((nr.gated_mlp(x, W_in, W_out)[:n], 128), (nr.gated_mlp(x[:n], W_in, W_out), n),
                  (nr.gated_mlp(x[:n], W_in, W_out, keep=True)[0], n)):
        assert float((y.double() - exact).norm()) <= (1.01 if of <= 16 else 1.7 if n == 1 else 1.5) * once


@pytest.mark.parametrize("n", [1, 2, 5, 12, 16])
@pytest.mark.parametrize("d,f", [(64, 128), (77, 301), (128, 192), (264, 515)])
def test_few_rows_are_rounded_once(n, d, f):
    """Two planes leave 2^-16 of m, dL/da and dL/db, 2^-8 of a rounding: results are as far off
    as rounding the exact ones, to a percent."""
    x, W_in, W_out, g = inputs(n, d, f, torch.bfloat16, seed=n + f)
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    got = (y, *nr.gated_mlp_backward(x, W_in, W_out, kept, g))
    ref = reference(x, W_in, W_out, g)[::2]
    for name, v, r in zip(("y", "gx", "gW_in", "gW_out"), got, ref):
        once = float((r.to(torch.bfloat16).double() - r).norm())
        assert float((v.double() - r).norm()) <= 1.02 * once, name


def test_infinities_of_few_rows():
    """A row with an infinite product leaves the others alone, in both directions."""
    x, W_in, W_out, g = inputs(16, 64, 128, torch.bfloat16, seed=2)
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    gx = nr.gated_mlp_backward(x, W_in, W_out, kept, g)[0]
    x2 = x.clone()
    x2[7], x2[13] = float("inf"), float("nan")
    y2, kept2 = nr.gated_mlp(x2, W_in, W_out, keep=True)
    gx2 = nr.gated_mlp_backward(x2, W_in, W_out, kept2, g)[0]
    live = [i for i in range(16) if i not in (7, 13)]
    assert torch.equal(y[live], y2[live]) and torch.equal(gx[live], gx2[live])
    assert bool(y2[13].isnan().all()) and not bool(y2[7].isfinite().any())


def test_what_is_kept_tells_numbers_of_rows_apart():
    size = nr.load().nrnn_gated_mlp_kept_bytes
    for dtype in (0, 1):
        for f in (1, 8, 100, 4096):
            sizes = [size(n, f, dtype) for n in range(400)]
            assert len(set(sizes)) == 400
