"""GPU parity of the language-model operators against plain float64.

Tolerances, element by element, with u = 2^-24 (fp32, 24 significant bits) and
rounding to bf16 of at most 2^-8 relative (8 significant bits):
  * sums of n products or values in fp32 in any order: n u of the sum of the
    magnitudes at worst; the tests allow the small constant each case names;
  * the tensor cores' fp32 accumulation may drop bits below the accumulator's
    last: one step of 16 products costs up to 2 u of the running magnitude;
  * ex2, rcp and rsqrt approximations: a few 2^-22 relative;
  * a bf16 result adds 2^-8 of its own value."""
import math

import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = [torch.float32, torch.bfloat16]
EPS = 1e-6


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, t=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)


def round_tol(t):
    return 2.0 ** -8 if t == torch.bfloat16 else 0.0


def check(got, ref, tol, what=""):
    """|got - ref| <= tol element by element; NaN nowhere it is not in ref."""
    got = got.to(F64)
    assert got.shape == ref.shape
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - ref).abs().max()),
                                 float((tol if torch.is_tensor(tol) else torch.tensor(tol)).min()))


# ------------------------------------------------------------------ embedding
EMBED = [(1, 1, 1), (1, 5, 8), (31, 7, 3), (32, 50, 64), (33, 50, 250), (65, 40000, 128),
         (1000, 300, 515), (4097, 33, 1024), (20000, 65536, 256), (9000, 262145, 40)]


def embed_inputs(n, V, d, t, seed, idt):
    g = gen(seed)
    ids = torch.randint(0, V, (n,), generator=g, device="cuda")
    ids[torch.rand(n, generator=g, device="cuda") < 0.3] = V // 2      # one id that spans many chunks
    return g, ids.to(idt)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,V,d", EMBED)
def test_embedding(n, V, d, t):
    g, ids = embed_inputs(n, V, d, t, 1, torch.int64 if n % 2 else torch.int32)
    W = randn(g, V, d, t=t)
    got = nr.embedding(ids, W, scale=1.7, padding_idx=V - 1)
    ref = (W[ids.long()].float() * 1.7).to(t)     # one fp32 product, one rounding: equal bit by bit
    ref[ids.long() == V - 1] = 0
    assert torch.equal(got, ref)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,V,d", EMBED)
def test_embedding_backward(n, V, d, t):
    g, ids = embed_inputs(n, V, d, t, 2, torch.int32 if n % 2 else torch.int64)
    go = randn(g, n, d, t=t)
    pad = V - 1 if V > 1 else None
    got = nr.embedding_backward(ids, go, V, scale=0.3, padding_idx=pad)
    live = ids.long() != (V - 1 if V > 1 else -1)
    k = ids.long()[live]
    s = float(torch.tensor(0.3, dtype=torch.float32))
    ref = torch.zeros(V, d, device="cuda", dtype=F64).index_add_(0, k, go[live].to(F64) * s)
    mag = torch.zeros(V, d, device="cuda", dtype=F64).index_add_(0, k, go[live].to(F64).abs() * s)
    # sums in groups of 32 and of chunks: under 32 + n / 32 + 32 additions deep
    depth = 64 + n / 32
    check(got, ref, depth * 2.0 ** -24 * mag + round_tol(t) * ref.abs())
    again = nr.embedding_backward(ids, go, V, scale=0.3, padding_idx=pad)
    assert torch.equal(got, again)                # the order of the sums is fixed
    # added to a given gradient: one more rounding, rows of absent ids untouched
    base = randn(g, V, d, t=t)
    acc = nr.embedding_backward(ids, go, V, scale=0.3, padding_idx=pad, out=base.clone(), accumulate=True)
    sum_ref = base.to(F64) + ref
    check(acc, sum_ref, depth * 2.0 ** -24 * (mag + base.to(F64).abs()) + round_tol(t) * sum_ref.abs())
    absent = torch.ones(V, dtype=torch.bool, device="cuda")
    absent[k] = False
    assert torch.equal(acc[absent], base[absent])


def test_embedding_edges():
    W = randn(gen(3), 10, 24)
    ids = torch.tensor([[3, -1, 10], [9, 2 ** 40, 0]], device="cuda")
    out = nr.embedding(ids, W)
    assert out.shape == (2, 3, 24)
    bad = torch.tensor([[False, True, True], [False, True, False]], device="cuda")
    assert bool(out[bad].isnan().all()) and torch.equal(out[~bad], W[ids[~bad]])
    # ids outside the vocabulary and padding take no part in the gradient, whatever they hold
    g = torch.ones(2, 3, 24, device="cuda")
    g[bad] = float("nan")
    gW = nr.embedding_backward(ids, g, 10)
    ref = torch.zeros(10, 24, device="cuda")
    ref[[3, 9, 0]] = 1
    assert torch.equal(gW, ref)
    assert nr.embedding(ids[:0], W).shape == (0, 3, 24)
    assert torch.equal(nr.embedding_backward(ids[:0], g[:0], 10), torch.zeros(10, 24, device="cuda"))
    all_pad = torch.full((100,), 4, device="cuda")
    assert torch.equal(nr.embedding(all_pad, W, padding_idx=4), torch.zeros(100, 24, device="cuda"))
    gp = torch.full((100, 24), float("inf"), device="cuda")
    assert torch.equal(nr.embedding_backward(all_pad, gp, 10, padding_idx=4), torch.zeros(10, 24, device="cuda"))


def test_embedding_strides_and_alignment():
    g = gen(4)
    big = randn(g, 50, 65, t=torch.bfloat16)
    ids = torch.randint(0, 50, (40, 2), generator=g, device="cuda")[:, 0]
    W = big[:, 1:]                                   # strided: copied
    assert torch.equal(nr.embedding(ids, W), W[ids])
    flat = randn(g, 50 * 64 + 1, t=torch.bfloat16)[1:].view(50, 64)   # 2-byte aligned rows
    assert torch.equal(nr.embedding(ids, flat), flat[ids])
    a = nr.embedding_backward(ids, flat[:40], 50)
    assert torch.equal(a, nr.embedding_backward(ids, flat[:40].clone(), 50))


def test_embedding_rows_beyond_32_bit_offsets():
    V, d = 2_200_000, 1024                          # 2.25e9 elements
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, V - 2, V - 1], device="cuda")
    W[V - 1] = 3
    W[V - 2] = 2
    out = nr.embedding(ids, W)
    assert torch.equal(out[:, 0].float(), torch.tensor([3.0, 0, 2, 3], device="cuda"))
    del W
    gW = nr.embedding_backward(ids, out, V)
    assert float(gW[V - 1].float().min()) == 6 and float(gW[V - 2].float().max()) == 2
    assert int((gW[:V - 2] != 0).sum()) == 0


# ----------------------------------------------------------------- block norm
NORM = [(1, 1), (2, 7), (5, 64), (17, 65), (33, 250), (64, 256), (40, 515), (300, 512), (21, 1024),
        (9, 1032), (3, 4096), (5, 8191), (4, 8192)]


def norm_inputs(n, d, t, gate, seed):
    g = gen(seed)
    x, h = randn(g, n, d, t=t, std=2.0), randn(g, n, d, t=t, std=0.4)
    gt = randn(g, n, d, t=t) if gate else None
    w = [1 + randn(g, d, std=0.1) for _ in range(3)]
    return g, x, h, gt, w


def rms64(v):
    r = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    return v * r, r


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d", NORM)
def test_block_norm(n, d, t, gate):
    g, x, h, gt, w = norm_inputs(n, d, t, gate, 5)
    x_out, u = nr.block_norm(x, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2], eps=EPS)
    hn, _ = rms64(h.to(F64))
    y = hn * w[0].to(F64)
    if gate:
        y = y * torch.nn.functional.silu(gt.to(F64))
    xr = x.to(F64) + w[1].to(F64) * y
    xn, r = rms64(xr)
    ur = xn * w[2].to(F64)
    # a handful of fp32 operations and approximations: 2^-20 of the magnitudes
    ex = 2.0 ** -20 * (x.to(F64).abs() + (w[1].to(F64) * y).abs() * 4)
    check(x_out, xr, ex + round_tol(t) * xr.abs(), "x_out")
    eu = r * w[2].to(F64).abs() * ex + 2.0 ** -19 * ur.abs() + ur.abs() * r * (ex.square().mean(-1, keepdim=True).sqrt())
    check(u, ur, eu + round_tol(t) * ur.abs(), "u")
    # without the next norm, in place, and the norm alone
    alone, none = nr.block_norm(x, h=h, gate=gt, w_post=w[0], scale=w[1], eps=EPS, next_norm=False)
    assert none is None and torch.equal(alone, x_out)
    mine = x.clone()
    same, u2 = nr.block_norm(mine, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2], eps=EPS, out=mine)
    assert same is mine and torch.equal(mine, x_out) and torch.equal(u2, u)
    first, u3 = nr.block_norm(x, w_pre=w[2], eps=EPS)
    assert first.data_ptr() == x.data_ptr()
    nx, _ = rms64(x.to(F64))
    check(u3, nx * w[2].to(F64), (2.0 ** -19 + round_tol(t)) * (nx * w[2].to(F64)).abs(), "norm alone")


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,d", NORM + [(2600, 64), (3001, 250)])
def test_block_norm_backward(n, d, t, gate):
    g, x, h, gt, w = norm_inputs(n, d, t, gate, 6)
    g_x, g_u = randn(g, n, d, t=t, std=0.1), randn(g, n, d, t=t, std=0.1)
    got = nr.block_norm_backward(x, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2], g_x=g_x, g_u=g_u, eps=EPS)
    W = [v.to(F64) for v in w]
    xn, r = rms64(x.to(F64))
    a = g_u.to(F64) * W[2]
    gx = g_x.to(F64) + r * (a - xn * (a * xn).mean(-1, keepdim=True))
    hn, q = rms64(h.to(F64))
    if gate:
        z = gt.to(F64)
        s = torch.sigmoid(z)
        of, slope = z * s, s * (1 + z * (1 - s))
    else:
        of, slope = torch.ones_like(hn), None
    gy = gx * W[1]
    b = gy * of * W[0]
    gh = q * (b - hn * (b * hn).mean(-1, keepdim=True))
    k = 2.0 ** -19
    # magnitudes before the cancellations of each formula
    mx = g_x.to(F64).abs() + r * (a.abs() + xn.abs() * (a * xn).abs().mean(-1, keepdim=True))
    my = mx * W[1].abs() * (of.abs() + 2.0 ** -3)          # silu near 0 is z / 2 with s approximate
    mb = my * W[0].abs()
    mh = q * (mb + hn.abs() * (mb * hn.abs()).mean(-1, keepdim=True))
    rt = round_tol(t)
    check(got.gx, gx, k * mx + rt * gx.abs(), "gx")
    check(got.gh, gh, k * mh + rt * gh.abs(), "gh")
    if gate:
        gg = gy * hn * W[0] * slope
        check(got.g_gate, gg, k * (mx * (W[1] * hn * W[0]).abs() * 1.2) + rt * gg.abs(), "g_gate")
    else:
        assert got.g_gate is None
    depth = (k + (64 + n / 608) * 2.0 ** -24)
    check(got.gw_post, (gy * of * hn).sum(0), depth * (my * hn.abs()).sum(0), "gw_post")
    check(got.g_scale, (gx * hn * W[0] * of).sum(0), depth * (mx * (hn * W[0]).abs() * (of.abs() + 2.0 ** -3)).sum(0), "g_scale")
    check(got.gw_pre, (g_u.to(F64) * xn).sum(0), depth * (g_u.to(F64) * xn).abs().sum(0), "gw_pre")
    again = nr.block_norm_backward(x, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2], g_x=g_x, g_u=g_u, eps=EPS)
    for p, o in zip(got, again):
        assert (p is None and o is None) or torch.equal(p, o)


def test_block_norm_backward_parts():
    """g_x alone, g_u alone and the norm alone agree with the full call fed zeros."""
    g, x, h, gt, w = norm_inputs(50, 96, torch.float32, True, 7)
    kw = dict(h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2])
    ga = randn(g, 50, 96)
    zero = torch.zeros_like(ga)
    only_x, full_x = nr.block_norm_backward(x, g_x=ga, **kw), nr.block_norm_backward(x, g_x=ga, g_u=zero, **kw)
    assert only_x.gw_pre is None and bool((full_x.gw_pre == 0).all())
    only_u, full_u = nr.block_norm_backward(x, g_u=ga, **kw), nr.block_norm_backward(x, g_x=zero, g_u=ga, **kw)
    for p, o in zip(only_x[:5], full_x[:5]):
        assert torch.equal(p, o)
    for p, o in zip(only_u, full_u):
        assert torch.equal(p, o)
    alone = nr.block_norm_backward(x, w_pre=w[2], g_u=ga)
    assert alone.gh is None and alone.g_scale is None
    assert torch.equal(alone.gx, only_u.gx) and torch.equal(alone.gw_pre, only_u.gw_pre)
    # weights left out are ones
    ones = torch.ones(96, device="cuda")
    p = nr.block_norm_backward(x, h=h, gate=gt, g_x=ga, g_u=ga)
    o = nr.block_norm_backward(x, h=h, gate=gt, w_post=ones, scale=ones, w_pre=ones, g_x=ga, g_u=ga)
    for v, e in zip(p, o):
        assert torch.equal(v, e)


def test_block_norm_edges():
    x = torch.zeros(3, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    x_out, u = nr.block_norm(x, h=x, w_post=w)
    assert bool((x_out == 0).all()) and bool((u == 0).all())           # rows of zeros
    g = nr.block_norm_backward(x, h=x, g_x=x + 1, g_u=x + 1)
    assert all(bool(v.isfinite().all()) for v in g if v is not None)
    empty = torch.empty(0, 40, device="cuda")
    a, b = nr.block_norm(empty, h=empty)
    assert a.shape == b.shape == (0, 40)
    g = nr.block_norm_backward(empty, h=empty, g_x=empty, g_u=empty)
    assert g.gx.shape == (0, 40) and bool((g.gw_post == 0).all()) and bool((g.gw_pre == 0).all())
    # a row that holds NaN or infinity stays alone
    x = randn(gen(8), 5, 64)
    bad = x.clone()
    bad[2, 3], bad[4, 0] = float("nan"), float("inf")
    good, _ = nr.block_norm(x, h=x)
    got, u = nr.block_norm(bad, h=bad)
    assert torch.equal(got[[0, 1, 3]], good[[0, 1, 3]])
    assert bool(u[2].isnan().all()) and bool(u[4].isnan().any())
    # a gate far below or above zero
    gate = torch.tensor([-200.0, 200.0, 0.0], device="cuda").repeat(5, 22)[:, :64].contiguous()
    got, _ = nr.block_norm(x, h=x, gate=gate)
    hn, _ = rms64(x.to(F64))
    check(got, x.to(F64) + hn * gate.to(F64).clamp_min(0), 1e-4)


# ----------------------------------------------------------------- vocab loss
LOSS = [(1, 1, 1), (1, 300, 64), (2, 2, 3), (5, 1000, 65), (127, 255, 8), (128, 256, 64), (129, 257, 72),
        (300, 5000, 515), (513, 3001, 1024), (2100, 700, 250), (700, 33000, 96)]


def loss_inputs(n, V, d, t, ignored, seed):
    g = gen(seed)
    x, W = randn(g, n, d, t=t), randn(g, V, d, t=t, std=2 / math.sqrt(d))
    target = torch.randint(0, V, (n,), generator=g, device="cuda")
    if ignored:
        target[torch.rand(n, generator=g, device="cuda") < ignored] = -100
        x[target == -100] = float("nan")      # what ignored rows hold reaches nothing
    return g, x, W, target, randn(g, n)


def loss64(x, W, target, gl, c):
    kept = target != -100
    X = torch.where(kept[:, None], x.to(F64), 0.0)
    z = c * X @ W.to(F64).T
    lse = torch.logsumexp(z, 1)
    at = target.clamp_min(0)[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
    G = torch.exp(z - lse[:, None])
    G.scatter_add_(1, at, torch.full_like(lse[:, None], -1.0))
    G *= (torch.where(kept, gl.to(F64), 0.0) * c)[:, None]
    zmag = abs(c) * (X.abs() @ W.to(F64).abs().T).max(1).values
    return kept, X, torch.where(kept, lse, 0.0), loss, G, zmag


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,V,d", LOSS)
@pytest.mark.parametrize("ignored,c", [(0.0, 1.0), (0.3, 0.6)])
def test_vocab_loss(n, V, d, t, ignored, c):
    check_vocab_loss(n, V, d, t, ignored, c)


# few rows (4, 16 and 17: the edges of the fp32 few-rows form), rows too wide for it,
# more column tiles than pairs work side by side, a gradient cut into many parts,
# far fewer kept rows than rows, a vocabulary below one tile
MORE = [(4, 900, 96, 0.0), (16, 900, 515, 0.0), (16, 700, 1024, 0.4), (17, 900, 96, 0.0), (16, 300, 2600, 0.0),
        (200, 600, 2600, 0.1), (100, 50021, 512, 0.0), (3000, 2500, 320, 0.98), (5000, 40, 128, 0.5),
        (260, 20000, 1000, 0.0)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n,V,d,ignored", MORE)
def test_vocab_loss_more_shapes(n, V, d, ignored, t):
    check_vocab_loss(n, V, d, t, ignored, 0.8)


def check_vocab_loss(n, V, d, t, ignored, c):
    g, x, W, target, gl = loss_inputs(n, V, d, t, ignored, 9)
    idt = torch.int32 if n % 2 else torch.int64
    loss, lse = nr.vocab_loss(x, W, target.to(idt), logit_scale=c)
    kept, X, lse_ref, loss_ref, G, zmag = loss64(x, W, target, gl, c)
    # logits: up to d / 16 accumulation steps of 2 u (d <= 2600: 2^-15.6, here with
    # errors that do not all lie one way 2^-17); then sums of positive terms
    tz = 2.0 ** -17 * zmag + 2.0 ** -20 * (1 + lse_ref.abs())
    check(lse, lse_ref, tz, "lse")
    check(loss, loss_ref, 2 * tz, "loss")
    assert bool((loss[~kept] == 0).all()) and bool((lse[~kept] == 0).all())
    gx, gW = nr.vocab_loss_backward(x, W, target.to(idt), lse, gl, logit_scale=c)
    # p is off by tz relative; G's rounding to bf16 (2^-8) where inputs are bf16,
    # or 2^-16 for the fp32 products and their accumulation
    part = 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -16
    P = (G.abs() + gl.abs().to(F64)[:, None] * abs(c) * 2 * tz[:, None] * torch.where(kept, 1.0, 0.0)[:, None])
    rt = round_tol(t)
    gx_ref, gW_ref = G @ W.to(F64), G.T @ X
    check(gx, gx_ref, part * (G.abs() @ W.to(F64).abs()) + ((P - G.abs()) @ W.to(F64).abs()) + rt * gx_ref.abs(), "gx")
    check(gW, gW_ref, part * (G.abs().T @ X.abs()) + ((P - G.abs()).T @ X.abs()) + rt * gW_ref.abs(), "gW")
    assert bool((gx[~kept] == 0).all())
    again = nr.vocab_loss_backward(x, W, target.to(idt), lse, gl, logit_scale=c)
    assert torch.equal(gx, again[0]) and torch.equal(gW, again[1])


@pytest.mark.parametrize("t", TYPES)
def test_vocab_loss_edges(t):
    g, x, W, target, gl = loss_inputs(40, 500, 96, t, 0.0, 10)
    none = torch.full_like(target, -100)
    loss, lse = nr.vocab_loss(x * float("inf"), W, none)              # no row takes part
    assert bool((loss == 0).all()) and bool((lse == 0).all())
    gx, gW = nr.vocab_loss_backward(x * float("nan"), W, none, lse, gl)
    assert bool((gx == 0).all()) and bool((gW == 0).all())
    # a target outside the vocabulary: NaN in its row, nothing elsewhere
    wrong = target.clone()
    wrong[3], wrong[20] = 500, -7
    loss, lse = nr.vocab_loss(x, W, wrong)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[[3, 20]] = True
    good, _ = nr.vocab_loss(x, W, target)
    assert bool(loss[bad].isnan().all()) and torch.equal(loss[~bad], good[~bad])
    gx, gW = nr.vocab_loss_backward(x, W, wrong, lse, gl)
    assert bool(gx[bad].isnan().all()) and bool(gx[~bad].isfinite().all()) and bool(gW.isfinite().all())
    # ignore_index inside the vocabulary
    pad = torch.where(torch.arange(40, device="cuda") % 3 == 0, 0, target)
    loss, lse = nr.vocab_loss(x, W, pad, ignore_index=0)
    assert bool((loss[::3] == 0).all())
    # no rows at all
    loss, lse = nr.vocab_loss(x[:0], W, target[:0])
    assert loss.shape == (0,)
    gx, gW = nr.vocab_loss_backward(x[:0], W, target[:0], lse, gl[:0])
    assert gx.shape == (0, 96) and bool((gW == 0).all())
    # a kept row that holds NaN gives NaN in its own row only
    xn = x.clone()
    xn[5, 7] = float("nan")
    loss, _ = nr.vocab_loss(xn, W, target)
    assert bool(loss[5].isnan()) and torch.equal(loss[:5], good[:5]) and torch.equal(loss[6:], good[6:])
    # leading dimensions
    l2, s2 = nr.vocab_loss(x.view(4, 10, 96), W, target.view(4, 10))
    assert l2.shape == (4, 10) and torch.equal(l2.reshape(-1), good)


def test_vocab_loss_large_logits():
    """Logits of several thousands: the running maximum keeps the sums finite."""
    g, x, W, target, gl = loss_inputs(64, 3000, 128, torch.float32, 0.0, 11)
    loss, lse = nr.vocab_loss(x, W, target, logit_scale=500.0)
    kept, X, lse_ref, loss_ref, G, zmag = loss64(x, W, target, gl, 500.0)
    tz = 2.0 ** -17 * zmag + 2.0 ** -20 * (1 + lse_ref.abs())
    check(lse, lse_ref, tz)
    check(loss, loss_ref, 2 * tz)
    loss, lse = nr.vocab_loss(x, W, target, logit_scale=-1.0)
    kept, X, lse_ref, loss_ref, G, zmag = loss64(x, W, target, gl, -1.0)
    check(loss, loss_ref, 2.0 ** -16 * zmag + 2.0 ** -19 * (1 + lse_ref.abs()))
    loss, lse = nr.vocab_loss(x, W, target, logit_scale=0.0)
    check(loss, torch.full_like(loss_ref, math.log(3000)), 1e-5)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [4, 40])
def test_vocab_loss_lowest_value(n, t):
    """A vocabulary row that the type's lowest value masks takes no probability."""
    g, x, W, target, gl = loss_inputs(n, 500, 96, t, 0.0, 14)
    target.clamp_min_(1)
    x[:, 0] = 0.5
    x[1, 1] = torch.finfo(t).max
    W[:, 1] = 0
    W[0] = 0
    W[0, 0] = torch.finfo(t).min
    loss, lse = nr.vocab_loss(x, W, target)
    x2 = x.clone()
    x2[1, 1] = 0
    kept, X, lse_ref, loss_ref, G, zmag = loss64(x2, W[1:], target - 1, gl, 1.0)
    tz = 2.0 ** -17 * zmag + 2.0 ** -20 * (1 + lse_ref.abs())
    check(lse, lse_ref, tz, "lse")
    check(loss, loss_ref, 2 * tz, "loss")
    gx, gW = nr.vocab_loss_backward(x2, W, target, lse, gl)
    part = 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -16
    more = gl.abs().to(F64)[:, None] * 2 * tz[:, None] + part * G.abs()
    gx_ref, gW_ref, rt = G @ W[1:].to(F64), G.T @ X, round_tol(t)
    check(gx, gx_ref, more @ W[1:].to(F64).abs() + rt * gx_ref.abs(), "gx")
    check(gW[1:], gW_ref, more.T @ X.abs() + rt * gW_ref.abs(), "gW")
    assert bool((gW[0] == 0).all())


def test_vocab_loss_strides_and_alignment():
    g, x, W, target, gl = loss_inputs(60, 700, 64, torch.bfloat16, 0.2, 12)
    flat = torch.empty(700 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(700, 64).copy_(W)
    loss, lse = nr.vocab_loss(x, W, target)
    assert flat.data_ptr() % 16 != 0
    l2, s2 = nr.vocab_loss(x.t().contiguous().t(), flat, target)
    assert torch.equal(loss, l2)
    a, b = nr.vocab_loss_backward(x, W, target, lse, gl), nr.vocab_loss_backward(x, flat, target, lse, gl)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_vocab_loss_pieces_of_a_long_vocabulary():
    """More than one piece of G: rows x V above the workspace's piece, and rows
    of W and gW beyond 32-bit offsets."""
    n, V, d = 6, 2_200_000, 1024
    g = gen(13)
    x = randn(g, n, d, t=torch.bfloat16, std=0.05)
    W = torch.zeros(V, d, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 5000, V // 2, V - 2, V - 1], device="cuda")
    W[at] = randn(g, n, d, t=torch.bfloat16, std=0.5)
    loss, lse = nr.vocab_loss(x, W, at)
    z = x.to(F64) @ W[at].to(F64).T
    lse_ref = torch.log(torch.exp(z).sum(1) + (V - n))
    check(lse, lse_ref, 1e-4)
    check(loss, lse_ref - z.diagonal(), 1e-4)
    gx, gW = nr.vocab_loss_backward(x, W, at, lse, torch.ones(n, device="cuda"))
    G = torch.exp(z - lse_ref[:, None]) - torch.eye(n, device="cuda", dtype=F64)
    check(gx, G @ W[at].to(F64), 2.0 ** -8 * (G.abs() @ W[at].to(F64).abs()) + 1e-6)
    check(gW[at], G.T @ x.to(F64), 2.0 ** -8 * (G.abs().T @ x.to(F64).abs()) + 1e-6)


def test_vocab_loss_many_rows_in_pieces():
    """Rows enough for several pieces of the vocabulary, checked on sampled rows."""
    n, V, d = 150_000, 9000, 64
    g, x, W, target, gl = loss_inputs(n, V, d, torch.bfloat16, 0.1, 14)
    gl = gl / n
    loss, lse = nr.vocab_loss(x, W, target)
    gx, gW = nr.vocab_loss_backward(x, W, target, lse, gl)
    some = torch.cat([torch.arange(200, device="cuda"), torch.arange(n - 200, n, device="cuda")])
    kept, X, lse_ref, loss_ref, G, zmag = loss64(x[some], W, target[some], gl[some], 1.0)
    tz = 2.0 ** -17 * zmag + 2.0 ** -20 * (1 + lse_ref.abs())
    check(lse[some], lse_ref, tz)
    check(loss[some], loss_ref, 2 * tz)
    gx_ref = G @ W.to(F64)
    check(gx[some], gx_ref, (2.0 ** -8 + 2.0 ** -12) * (G.abs() @ W.to(F64).abs()) + 2.0 ** -8 * gx_ref.abs())
    ref = torch.zeros(V, d, device="cuda", dtype=F64)
    mag = torch.zeros(V, d, device="cuda", dtype=F64)
    for i in range(0, n, 10000):
        _, X, _, _, G, _ = loss64(x[i:i + 10000], W, target[i:i + 10000], gl[i:i + 10000], 1.0)
        ref += G.T @ X
        mag += G.abs().T @ X.abs()
    check(gW, ref, (2.0 ** -8 + 2.0 ** -12) * mag + 2.0 ** -8 * ref.abs())


# ---------------------------------------------------------------- differences
def test_gradients_against_differences():
    """Directional derivatives of the operators' own fp32 outputs by central
    differences: the step's square (third derivatives of order 10) and the
    outputs' rounding over the step bound the error."""
    g, x, W, target, gl = loss_inputs(60, 400, 80, torch.float32, 0.2, 15)
    x = torch.where(target[:, None] == -100, 0.0, x)
    lse = nr.vocab_loss(x, W, target)[1]
    gx, gW = nr.vocab_loss_backward(x, W, target, lse, gl)
    step = 1e-2
    for grad, move in ((gx, 0), (gW, 1)):
        to = randn(g, *grad.shape)
        to /= to.norm()

        def f(s):
            a, b = (x + s * to, W) if move == 0 else (x, W + s * to)
            return float((nr.vocab_loss(a, b, target)[0].double() * gl.double()).sum())
        num = (f(step) - f(-step)) / (2 * step)
        assert abs(num - float((grad.double() * to.double()).sum())) <= 10 * step ** 2 + 60 * 2.0 ** -20 / step
    g, x, h, gt, w = norm_inputs(20, 70, torch.float32, True, 16)
    a, b = randn(g, 20, 70), randn(g, 20, 70)
    x_out, _ = nr.block_norm(x, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2])
    r = nr.block_norm_backward(x_out, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2], g_x=a, g_u=b)
    args = dict(x=x, h=h, gate=gt, w_post=w[0], scale=w[1], w_pre=w[2])
    for name, grad in (("x", r.gx), ("h", r.gh), ("gate", r.g_gate), ("w_post", r.gw_post),
                       ("scale", r.g_scale), ("w_pre", r.gw_pre)):
        to = randn(g, *grad.shape)
        to /= to.norm()

        def f(s):
            o, u = nr.block_norm(**{**args, name: args[name] + s * to})
            return float((o.double() * a.double()).sum() + (u.double() * b.double()).sum())
        num = (f(step) - f(-step)) / (2 * step)
        assert abs(num - float((grad.double() * to.double()).sum())) <= 100 * step ** 2 + 60 * 2.0 ** -20 / step, name
    ids = torch.randint(0, 30, (100,), generator=g, device="cuda")
    W, go = randn(g, 30, 20), randn(g, 100, 20)
    gW = nr.embedding_backward(ids, go, 30, scale=2.0)
    to = randn(g, 30, 20)
    num = float(((nr.embedding(ids, W + to, scale=2.0) - nr.embedding(ids, W - to, scale=2.0)).double() * go.double()).sum()) / 2
    assert abs(num - float((gW.double() * to.double()).sum())) <= 2000 * 2.0 ** -20


# ------------------------------------------------------------------- refusals
def test_refusals():
    g = gen(17)
    x, ids = randn(g, 4, 16), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        nr.embedding(ids.float(), x)
    with pytest.raises(TypeError):
        nr.embedding(ids, x.half())
    with pytest.raises(ValueError):
        nr.embedding(ids, x[0])
    with pytest.raises(ValueError):
        nr.embedding_backward(ids[:3], x, 10)
    with pytest.raises(ValueError):
        nr.embedding_backward(ids, x, 0)
    with pytest.raises(ValueError):
        nr.embedding_backward(ids, x, 10, accumulate=True)
    with pytest.raises(ValueError):
        nr.embedding_backward(ids, x, 10, out=x)
    with pytest.raises(TypeError):
        nr.block_norm(randn(g, 2, 8200))
    with pytest.raises(ValueError):
        nr.block_norm(x, gate=x)
    with pytest.raises(ValueError):
        nr.block_norm(x, h=x[:2])
    with pytest.raises(ValueError):
        nr.block_norm(x, h=x, w_post=x[0, :8])
    with pytest.raises(ValueError):
        nr.block_norm(x, h=x, scale=x[0].bfloat16())
    with pytest.raises(ValueError):
        nr.block_norm(x, h=x, eps=-1.0)
    with pytest.raises(ValueError):
        nr.block_norm_backward(x, h=x)
    with pytest.raises(TypeError):
        nr.vocab_loss(x, x.bfloat16(), ids)
    with pytest.raises(ValueError):
        nr.vocab_loss(x, x[:, :8], ids)
    with pytest.raises(ValueError):
        nr.vocab_loss(x, x, ids[:2])
    loss, lse = nr.vocab_loss(x, x, ids)
    with pytest.raises(ValueError):
        nr.vocab_loss_backward(x, x, ids, lse.double(), lse)


def test_calls_on_another_stream():
    """Work on a side stream, ordered by events alone, gives the same results."""
    g, x, W, target, gl = loss_inputs(300, 2000, 128, torch.bfloat16, 0.1, 18)
    x = torch.where(target[:, None] == -100, 0.0, x.float()).to(x.dtype)
    ids = torch.randint(0, 2000, (300,), generator=g, device="cuda")

    def all_of():
        rows = nr.embedding(ids, W, scale=3.0)
        x_out, u = nr.block_norm(x, h=rows)
        loss, lse = nr.vocab_loss(u, W, target)
        gu, gW = nr.vocab_loss_backward(u, W, target, lse, gl)
        r = nr.block_norm_backward(x_out, h=rows, g_u=gu)
        nr.embedding_backward(ids, r.gh, 2000, scale=3.0, out=gW, accumulate=True)
        return loss, gu, r.gx, gW
    ref = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_of()
    torch.cuda.current_stream().wait_stream(side)
    for p, o in zip(ref, got):
        assert torch.equal(p, o)


def test_capture_in_a_graph():
    """The calls launch on the current stream only and never synchronise."""
    g, x, W, target, gl = loss_inputs(200, 1500, 64, torch.bfloat16, 0.0, 19)
    loss, lse = nr.vocab_loss(x, W, target)
    ref = nr.vocab_loss_backward(x, W, target, lse, gl)
    ids = target.clone()
    ref_e = nr.embedding_backward(ids, ref[0], 1500)
    ref_n = nr.block_norm_backward(x, h=x, g_x=ref[0], g_u=ref[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l2, s2 = nr.vocab_loss(x, W, target)
        got = nr.vocab_loss_backward(x, W, target, s2, gl)
        got_e = nr.embedding_backward(ids, got[0], 1500)
        got_n = nr.block_norm_backward(x, h=x, g_x=got[0], g_u=got[0])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, l2) and torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    assert torch.equal(ref_e, got_e) and torch.equal(ref_n.gw_pre, got_n.gw_pre)
