"""The norms on tensors that do not share an alignment: rows taken by elements, by teams
of every size.  Formulas and bounds as for aligned tensors: a handful of fp32 operations
and approximations, 2^-19 of the magnitudes before each formula's cancellations; sums
over the rows as deep as a team's rows and the joins; a bf16 result rounded by 2^-8."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64
EPS = 1e-6


def moved(v):
    """The same values one element further on in memory."""
    out = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)[1:].view(v.shape).copy_(v)
    assert out.data_ptr() % 16 and out.is_contiguous()
    return out


def check(got, ref, tol, what):
    bad = ~((got.to(F64) - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got.to(F64) - ref).abs().max()))


@pytest.mark.parametrize("which", ["x", "h", "gate", "all"])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(1, 1), (700, 3), (300, 24), (501, 96), (64, 256), (333, 300), (40, 1000), (5, 4096), (3, 8190)])
def test_norms_of_moved_tensors(n, d, t, which):
    g = torch.Generator(device="cuda")
    g.manual_seed(71)

    def randn(*s, std=1.0, t=t):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(t)
    v = {"x": randn(n, d, std=2.0), "h": randn(n, d, std=0.4), "gate": randn(n, d)}
    g_x, g_u = randn(n, d, std=0.1), randn(n, d, std=0.1)
    w = [1 + randn(d, std=0.1, t=torch.float32) for _ in range(3)]
    for k in v:
        if which in (k, "all"):
            v[k] = moved(v[k])
    if which == "all":
        g_x, g_u = moved(g_x), moved(g_u)
    rt, k = (2.0 ** -8 if t == torch.bfloat16 else 0.0), 2.0 ** -19
    x, h, z = (v[name].to(F64) for name in ("x", "h", "gate"))
    W = [u.to(F64) for u in w]
    q = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    hn, s = h * q, torch.sigmoid(z)
    of, slope = z * s, s * (1 + z * (1 - s))
    y = hn * W[0] * of
    xr = x + W[1] * y
    r = torch.rsqrt(xr.square().mean(1, keepdim=True) + EPS)
    x_out, u = nr.block_norm(v["x"], h=v["h"], gate=v["gate"], w_post=w[0], scale=w[1], w_pre=w[2], eps=EPS)
    ex = k * (x.abs() + (W[1] * y).abs() * 4)
    check(x_out, xr, ex + rt * xr.abs(), "x_out")
    ur = xr * r * W[2]
    eu = r * W[2].abs() * ex + k * ur.abs() + ur.abs() * r * ex.square().mean(1, keepdim=True).sqrt()
    check(u, ur, eu + rt * ur.abs(), "u")

    got = nr.block_norm_backward(v["x"], h=v["h"], gate=v["gate"], w_post=w[0], scale=w[1], w_pre=w[2], g_x=g_x, g_u=g_u, eps=EPS)
    r = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    xn, a, ga = x * r, g_u.to(F64) * W[2], g_x.to(F64)
    gx = ga + r * (a - xn * (a * xn).mean(1, keepdim=True))
    b = gx * W[1] * of * W[0]
    gh = q * (b - hn * (b * hn).mean(1, keepdim=True))
    mx = ga.abs() + r * (a.abs() + xn.abs() * (a * xn).abs().mean(1, keepdim=True))
    mof = of.abs() + 2.0 ** -3
    mb = mx * W[1].abs() * mof * W[0].abs()
    mh = q * (mb + hn.abs() * (mb * hn.abs()).mean(1, keepdim=True))
    check(got.gx, gx, k * mx + rt * gx.abs(), "gx")
    check(got.gh, gh, k * mh + rt * gh.abs(), "gh")
    gg = gx * W[1] * hn * W[0] * slope
    check(got.g_gate, gg, k * mx * (W[1] * hn * W[0]).abs() * 1.2 + rt * gg.abs(), "g_gate")
    depth = k + (64 + n / 608) * 2.0 ** -24
    check(got.gw_post, (gx * W[1] * of * hn).sum(0), depth * (mx * W[1].abs() * mof * hn.abs()).sum(0), "gw_post")
    check(got.g_scale, (gx * hn * W[0] * of).sum(0), depth * (mx * (hn * W[0]).abs() * mof).sum(0), "g_scale")
    check(got.gw_pre, (g_u.to(F64) * xn).sum(0), depth * (g_u.to(F64) * xn).abs().sum(0), "gw_pre")


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,d", [(700, 3), (300, 24), (333, 300), (5, 4097)])
def test_norms_of_moved_tensors_in_place(n, d, t):
    g = torch.Generator(device="cuda")
    g.manual_seed(72)
    x, h = (torch.randn(n, d, generator=g, device="cuda").to(t) for _ in range(2))
    for place in (x.clone(), moved(x)):
        ref = nr.block_norm(place, h=h)
        same, u = nr.block_norm(place, h=h, out=place)
        assert same is place and torch.equal(place, ref[0]) and torch.equal(u, ref[1])
