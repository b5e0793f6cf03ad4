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


@pytest.mark.parametrize("n", [1, 8, 16, 17])
def test_what_differs_by_the_rows_beside(n):
    """A bf16 row's y is rounded once where at most 16 rows keep nothing, and m before it
    otherwise: within 1.5 roundings of one another normwise (sqrt(2) and chance)."""
    x, W_in, W_out, _ = inputs(64, 256, 512, torch.bfloat16, seed=3)
    many, few = nr.gated_mlp(x, W_in, W_out)[:n].double(), nr.gated_mlp(x[:n], W_in, W_out).double()
    kept = nr.gated_mlp(x[:n], W_in, W_out, keep=True)[0].double()
    exact = reference(x[:n], W_in, W_out)[0]
    once = float((exact.to(torch.bfloat16).double() - exact).norm())
    assert torch.equal(many, kept)
    assert float((many - exact).norm()) <= (1.7 if n == 1 else 1.5) * once    # (one row: 256 results)
    assert float((few - exact).norm()) <= (1.01 if n <= 16 else 1.5) * once
