"""How exact the gated feed-forward block's training step is, from what it rounds.

With a = x Wg^T, b = x Wu^T, s = sig(a) the forward keeps p = dm/da = b (s + a s (1 - s)) and
q = dm/db = a s: in fp32, or for bf16 without the low 8 of their 32 bits.  bf16 rounds
m = q b, ga = gm p and gb = gm q once each, as the operands of the next product, and the
results once.

Normwise: a value's rounding to bf16 is an error of its own, so one of the operand and one of
the result add up to sqrt(2) of what rounding the exact result leaves; a third one, of p or q,
would make it sqrt(3).  Sums over 64 and more products and tens of thousands of results leave
a few percent of chance: 1.5 at most."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = [torch.float32, torch.bfloat16]


def inputs(n, d, f, t, seed, gate_scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std
    W_in = randn(2 * f, d, std=d ** -0.5)
    W_in[:f] *= gate_scale
    return randn(n, d).to(t), W_in.to(t), randn(d, f, std=f ** -0.5).to(t), randn(n, d).to(t)


def results(x, W_in, W_out, g):
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    return dict(zip(("y", "gx", "gW_in", "gW_out"), (y, *nr.gated_mlp_backward(x, W_in, W_out, kept, g))))


def exact(x, W_in, W_out, g):
    x, W_in, W_out, g = (v.to(F64) for v in (x, W_in, W_out, g))
    a, b = (x @ W_in.T).chunk(2, 1)
    s = torch.sigmoid(a)
    m, gm = a * s * b, g @ W_out
    gab = torch.cat([gm * b * (s + a * s * (1 - s)), gm * a * s], 1)
    return {"y": m @ W_out.T, "gx": gab @ W_in, "gW_in": gab.T @ x, "gW_out": g.T @ m}


@pytest.mark.parametrize("n,d,f", [(64, 1024, 512), (300, 256, 1032), (1501, 250, 683), (4096, 512, 1024), (77, 1024, 2000)])
def test_bf16_results_are_two_roundings_off(n, d, f):
    data = inputs(n, d, f, torch.bfloat16, seed=n)
    got, ref = results(*data), exact(*data)
    for name, r in ref.items():
        once = float((r.to(torch.bfloat16).to(F64) - r).norm())
        off = float((got[name].to(F64) - r).norm())
        assert off <= 1.5 * once, (name, off / once)


def bounds(x, W_in, W_out, g):
    """Results and the largest their errors can be, element by element.

    A sum of K products is at most (K + 64) 2^-24 of their magnitudes off (fp32 sums in any
    order; the tensor cores' drop up to 2^-23 of the running magnitude a step of 16; fp32
    factors are split to 2^-24).  The exponent of a sigmoid is a log2(e), rounded to 2^-23 of
    its value, so that a falling sigmoid is |a| 2^-22 off, and the exponential and the
    reciprocal 2^-21; 1 - s is off by 2^-23 where s is next to one.  |silu''| is at most 0.5
    and (2 + |a|) exp(-|a|).  24 kept bits are at most 2^-15 off.  fp32's normal numbers end at
2^-126: a sigmoid below is zero (a = -665 at the scale of 3000), and any value or product may
be lost there, each by that much."""
    low = 2.0 ** -126
    t = x.dtype
    u, k = (2.0 ** -8, 2.0 ** -15) if t == torch.bfloat16 else (2.0 ** -24, 0.0)
    x, W_in, W_out, g = (v.to(F64) for v in (x, W_in, W_out, g))
    n, d = x.shape
    f = W_out.shape[1]

    def summed(K, magnitudes):
        return (K + 64) * 2.0 ** -24 * magnitudes + K * low

    def rounded(v, e):
        return e + u * (v.abs() + e) + low
    a, b = (x @ W_in.T).chunk(2, 1)
    ea, eb = summed(d, x.abs() @ W_in.abs().T).chunk(2, 1)
    s = torch.sigmoid(a)
    es = s * ((1 - s) * a.abs() * 2.0 ** -22 + 2.0 ** -21) + low
    q, rise = a * s, s + a * s * (1 - s)
    second = torch.minimum(torch.full_like(a, 0.5), (2 + a.abs() + ea) * torch.exp(ea - a.abs()))
    eq = 1.1 * ea + a.abs() * es + 2.0 ** -22 * q.abs()
    # |d(s + a s (1 - s)) / ds| <= 1 + |a| |1 - 2 s|, of which a s 2^-23 is left where s is next to one
    e_rise = second * ea + es * (1 + a.abs() * (1 - s)) + q.abs() * 2.0 ** -23 + 2.0 ** -22 * rise.abs()
    p, ep = b * rise, (b.abs() + eb) * e_rise + eb * rise.abs()
    m = q * b
    em = rounded(m, (b.abs() + eb) * eq + q.abs() * eb + 2.0 ** -23 * m.abs())
    ep, eq = ep + k * (p.abs() + ep), eq + k * (q.abs() + eq)
    y = m @ W_out.T
    ey = em @ W_out.abs().T + summed(f, m.abs() @ W_out.abs().T)
    gm = g @ W_out
    egm = summed(d, g.abs() @ W_out.abs())
    gab = torch.cat([gm * p, gm * q], 1)
    egab = torch.cat([egm * (p.abs() + ep) + gm.abs() * ep, egm * (q.abs() + eq) + gm.abs() * eq], 1)
    egab = rounded(gab, egab + 2.0 ** -23 * gab.abs())
    gx, gW_in, gW_out = gab @ W_in, gab.T @ x, g.T @ m
    return {"y": (y, rounded(y, ey)),
            "gx": (gx, rounded(gx, egab @ W_in.abs() + summed(2 * f, gab.abs() @ W_in.abs()))),
            "gW_in": (gW_in, rounded(gW_in, egab.T @ x.abs() + summed(n, gab.abs().T @ x.abs()))),
            "gW_out": (gW_out, rounded(gW_out, g.abs().T @ em + summed(n, g.abs().T @ m.abs())))}


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("scale", [1.0, 40.0, 3000.0, 1e-6])
@pytest.mark.parametrize("n,d,f", [(1, 8, 8), (3, 33, 7), (40, 64, 128), (31, 72, 17), (33, 250, 331), (300, 130, 514), (513, 96, 1032)])
def test_every_element(n, d, f, scale, t):
    data = inputs(n, d, f, t, seed=n + f, gate_scale=scale)
    got = results(*data)
    for name, (ref, tol) in bounds(*data).items():
        off = (got[name].to(F64) - ref).abs()
        assert bool((off <= tol).all()), (name, float((off / tol).max()), int((off > tol).sum()))


@pytest.mark.parametrize("t", TYPES)
def test_what_was_kept_before_does_not_matter(t):
    """The same results whatever the memory of kept and workspace held."""
    data = inputs(45, 40, 51, t, seed=1)
    ref = results(*data)
    x, W_in, W_out, g = data
    lib = nr.load()
    for fill in (0, 255):
        kept = torch.full((lib.nrnn_gated_mlp_kept_bytes(45, 51, 1 if t == torch.bfloat16 else 0),), fill, dtype=torch.uint8, device="cuda")
        ws = torch.full((1 << 24,), fill, dtype=torch.uint8, device="cuda")
        y = torch.empty_like(x)
        code = 1 if t == torch.bfloat16 else 0
        stream = torch.cuda.current_stream().cuda_stream
        assert lib.nrnn_gated_mlp_forward(x.data_ptr(), W_in.data_ptr(), W_out.data_ptr(), code, 45, 40, 51, y.data_ptr(),
                                          kept.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
        assert torch.equal(y, ref["y"])
        ws.fill_(fill)
        for v, name in zip(nr.gated_mlp_backward(x, W_in, W_out, kept, g, workspace=ws), ("gx", "gW_in", "gW_out")):
            assert torch.equal(v, ref[name]), name
