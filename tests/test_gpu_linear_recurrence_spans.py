"""The gated linear recurrence over sequences so long that a chain of few columns passes from
one span of 256 chunks (8192 steps in fp32, 16384 in bf16) to the next, with decays that
forget nothing on the way, against a float64 unroll.

Tolerances.  Falls are at most 2^-4, where a decay is one and its series: 2^-25 for that
addition and as much for the series.  A step rounds a sum and a product of decays by 2^-24
each; M_t = a M_{t-1} + |u| bounds what they are of, in any grouping.  u = s i v is 2^-20 of
its value off.  So E_t = a_t E_{t-1} + 3 2^-24 a_t M_{t-1} + 2^-20 |u_t|: under 1% of M after
40000 steps, where a carry that is lost or taken twice is of M's order.  The adjoint has the
same bound from the other end."""
import numpy as np
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

CASES = [(torch.float32, 1, [0, 25000]), (torch.float32, 3, [0, 16385]), (torch.bfloat16, 1, [0, 50001]), (torch.bfloat16, 2, [0, 33000]),
         # packs: a segment over three spans; heads beside a span's border; many short ones before and after
         (torch.float32, 1, [0, 100, 100, 700, 25000, 25001, 25001, 27000]), (torch.float32, 1, [0, 8192, 16384, 24576]),
         (torch.float32, 1, [0, 8191, 8193, 24570, 24570]), (torch.float32, 1, [*range(0, 9000, 500), 26000, *range(26100, 27000, 100)]),
         (torch.bfloat16, 1, [0, 16383, 49200, 49201, 50000]), (torch.bfloat16, 1, [0, 0, 40, 49999])]


def rounding(t):
    return 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24


def unroll(a, u, start):
    """h_t = a_t h_{t-1} + u_t with bounds: (h, M, E), each (T, d)."""
    h, M, E = (np.empty_like(a) for _ in range(3))
    x, m, e = start, np.abs(start), np.zeros_like(start)
    for t in range(len(a)):
        am = a[t] * m
        x, m, e = a[t] * x + u[t], am + np.abs(u[t]), a[t] * e + 3 * 2.0 ** -24 * am + 2.0 ** -20 * np.abs(u[t])
        h[t], M[t], E[t] = x, m, e
    return h, M, E


def check(got, want, tol, what):
    off = np.abs(got.double().cpu().numpy() - want)
    assert (off <= tol).all(), (what, float((off / tol).max()), int((off > tol).sum()), np.argwhere(off > tol)[:4].tolist())


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_chains_over_spans(case, given):
    t, B, bounds = CASES[case]
    d, T = 8, bounds[-1]
    pack = len(bounds) > 2
    g = torch.Generator(device="cuda")
    g.manual_seed(case)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std
    P = randn(B, T, 3 * d).to(t)
    # falls per step from 2^-4 down to 1e-6: memories of 16 steps and of a million
    rate = torch.tensor([0.06, 1e-2, 1e-3, 3e-4, 1e-4, 3e-5, 1e-5, 1e-6], device="cuda")
    params = torch.stack([rate, randn(d, std=0.5), randn(d, std=0.5)])
    seqs = [(0, s, e) for s, e in zip(bounds, bounds[1:])] if pack else [(b, 0, T) for b in range(B)]
    state = randn(len(seqs), d, std=3.0) if given else None
    gH = randn(B, T, d, std=0.1).to(t)
    g_last = randn(len(seqs), d, std=3.0) if given else None
    cu = torch.tensor(bounds, dtype=torch.int32) if pack else None
    H, last = nr.linear_recurrence(P, params, cu_seqlens=cu, state=state)
    got = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=cu, state=state, g_state=g_last)

    w, p = params.double().cpu().numpy(), P.double().cpu().numpy()
    r, i, v = 1 / (1 + np.exp(-(p[..., :d] + w[1]))), 1 / (1 + np.exp(-(p[..., d:2 * d] + w[2]))), p[..., 2 * d:]
    fall = w[0] * r
    a, s = np.exp(-fall), np.sqrt(-np.expm1(-2 * fall))
    Hn, gn, eps = H.double().cpu().numpy(), gH.double().cpu().numpy(), rounding(t)
    sums, offs = np.zeros((3, d)), np.zeros((3, d))
    for k, (b, t0, t1) in enumerate(seqs):
        at = (b, slice(t0, t1))
        start = state[k].double().cpu().numpy() if given else np.zeros(d)
        end = g_last[k].double().cpu().numpy() if given else np.zeros(d)
        if t0 == t1:
            assert torch.equal(last[k], state[k] if given else torch.zeros_like(last[k]))
            if given:
                assert torch.equal(got.g_state[k], g_last[k])
            continue
        h, _, E = unroll(a[at], s[at] * i[at] * v[at], start)
        check(H[at], h, E + eps * (np.abs(h) + E), ("H", k))
        check(last[k], h[-1], E[-1], ("last", k))
        # G_t = gH_t + a_{t+1} G_{t+1}, from the end of time; the last step's includes dL/dlast
        after = np.concatenate([a[at][1:], np.ones((1, d))])[::-1]
        G, _, EG = (x[::-1] for x in unroll(after, gn[at][::-1], end))
        before = np.concatenate([start[None], Hn[at][:-1]])
        own, new = a[at] * before, a[at] ** 2 / s[at] * i[at] * v[at]
        wr, fine = G * (own - new) * r[at], 2.0 ** -19 * np.abs(G) + EG
        d_wr = fine * (np.abs(own) + np.abs(new)) * r[at]
        factor = w[0] * (1 - r[at])
        ga, d_a = -wr * factor, d_wr * factor * (1 + 2.0 ** -19)
        gi, d_i = G * s[at] * v[at] * i[at] * (1 - i[at]), fine * s[at] * np.abs(v[at]) * i[at] * (1 - i[at])
        gv, d_v = G * s[at] * i[at], fine * s[at] * i[at]
        want, tol = np.concatenate([ga, gi, gv], 1), np.concatenate([d_a, d_i, d_v], 1)
        check(got.gP[at], want, tol + eps * (np.abs(want) + tol) + 2.0 ** -126, ("gP", k))
        if given:
            check(got.g_state[k], a[at][0] * G[0], EG[0] + 2.0 ** -23 * np.abs(G[0]), ("g_state", k))
        sums += np.stack([-wr.sum(0), ga.sum(0), gi.sum(0)])
        offs += np.stack([(d_wr + B * T * 2.0 ** -24 * np.abs(wr)).sum(0), (d_a + B * T * 2.0 ** -24 * np.abs(ga)).sum(0),
                          (d_i + B * T * 2.0 ** -24 * np.abs(gi)).sum(0)])
    check(got.gparams, sums, offs, "gparams")
