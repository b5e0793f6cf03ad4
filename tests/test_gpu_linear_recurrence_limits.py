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


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_states_of_constant_decays(t):
    """A decay that stays the same adds its error up 1 / (1 - a) times, and the states are fp32
    whatever the storage: decays of 2^z around the places where their series ends, after many
    steps and after one.

    Relative to h = u / (1 - a): 2^-25 of a's last addition and as much of its series, or 2^-22
    of the exponential; 2^-24 a step of the scan's own rounding; u is 2^-22 (exponential) times
    2 a^2 / (1 - a^2) / 2 off where 1 - a^2 is a difference, which begins at z = -0.18, and 2^-21
    for the square root and the gates besides."""
    d, T = 2048, 900
    z = torch.linspace(-0.4, -0.02, d, device="cuda", dtype=torch.float64)
    params = torch.zeros(3, d, device="cuda")
    params[0] = -z * 0.6931471805599453
    params[1:] = 60.0                                            # both gates open: r = i = 1
    P = torch.zeros(1, T, 3 * d, dtype=t, device="cuda")
    P[..., 2 * d:] = 1.0
    a = torch.exp(-params[0].double())
    u, steps = torch.sqrt(-torch.expm1(-2 * params[0].double())), torch.arange(1, T + 1, device="cuda").double()[:, None]
    h = u * -torch.expm1(-params[0].double() * steps) / -torch.expm1(-params[0].double())
    series = z > -0.18
    da = torch.where(series, 2.0 ** -24, 2.0 ** -22)
    du = 2.0 ** -21 + torch.where(series, 0.0, 2.0 ** -22 * a * a / (1 - a * a))
    tol = du + (da + 2.0 ** -24) / (1 - a)
    H, last = nr.linear_recurrence(P, params)
    for got, want, bound in ((last[0], h[-1], tol), (nr.linear_recurrence(P[:, :1], params)[1][0], h[0], du)):
        off = (got.double() - want).abs() / want
        assert bool((off <= bound).all()), (float((off / bound).max()), float(z[(off / bound).argmax()]), float(off.max()))
    assert torch.equal(H[0, -1], last[0].to(t))
