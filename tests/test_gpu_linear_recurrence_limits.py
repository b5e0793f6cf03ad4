"""The gated linear recurrence at rates next to zero: 1 - a^2 is then a subnormal number,
which counts as zero in both directions."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

#: a shut gate is bounded below by 2^-63, so that rate r runs from 1e-45 to 1e-36 (and over
#: fp32's least normal number, 1.2e-38); the last rates are subnormal themselves
RATES = [1e-26, 1e-24, 1e-22, 1e-21, 5e-20, 1e-19, 3e-19, 1e-17, 1e-45, 1e-40, 5e-39, 1.2e-38]


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T", [(1, 1), (1, 40), (2, 131), (130, 67)])
def test_rates_next_to_zero(B, T, t):
    """Everything is finite, and what has s or its square as a factor is as small as s.

    With rate r <= 1.1e-36 here, s <= 1.5e-18 and a is one, so the adjoint is the sum of gH
    and the last gradient after a step, at most T + 1.  Then |gP_v| and |gP_i| are at most
    (T + 1) s, and |gP_a| <= (T + 1) (|h| rate r + rate r / s): all below (T + 1) 1e-17, with
    |h| <= 1 + T s."""
    d = 8 * len(RATES)
    P = torch.zeros(B, T, 3 * d, device="cuda")
    gates = torch.tensor([-90.0, -45.0, -3e38, -200.0, -90.0, -44.0, -90.0, -60.0], device="cuda")   # shut
    P[..., :d] = gates.repeat(len(RATES))
    P[..., :d].view(B, T, len(RATES), 8)[:, :, 8:] = 3.0      # open, at the subnormal rates
    P[..., d:2 * d] = torch.tensor([0.0, 5.0, -90.0, 90.0], device="cuda").repeat(d // 4)
    P[:, ::2, 2 * d:] = 1.0                                    # v: zeros and ones
    P = P.to(t)
    rate = torch.tensor(RATES, device="cuda").repeat_interleave(8)
    params = torch.stack([rate, torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    state = torch.ones(B, d, device="cuda")
    H, last = nr.linear_recurrence(P, params, state=state)
    assert bool(((last - 1).abs() <= T * 2e-18 + 2.0 ** -23).all())
    gH = torch.ones(B, T, d, device="cuda", dtype=t)
    r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=state)
    for name, x in zip(("gP", "gparams", "g_state"), r):
        assert bool(x.isfinite().all()), name
    assert bool((r.gP.abs() <= (T + 1) * 1e-17).all())
    assert torch.equal(r.g_state, torch.full_like(state, T + 1))
