"""GPU parity of the gated linear recurrence against a float64 unroll.

Tolerances, element by element.  ex2, rcp and sqrt approximations and the roundings
around them leave a gate 2^-21 of its value off, and a decay exp(-fall) another
2^-21 fall; a step of the scan, in whatever order chunks are joined, adds a few 2^-24
of the magnitudes it adds.  So with c_t = (4 + 2 fall_t) 2^-21 a state is off by at
most E_t = a_t E_{t-1} + c_t (|a_t h_{t-1}| + |u_t|), and a result rounded to bf16 by
2^-8 of its value besides.  The backward's adjoint has the same bound in reverse."""
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


def rounding(t):
    return 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24


def check(got, ref, tol, what=""):
    got = got.to(F64)
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((got - ref).abs().max()), bad.nonzero()[:4].tolist())


def inputs(B, T, d, t, seed=0, std=1.0, fast=4.0):
    g = gen(seed)
    P = randn(g, B, T, 3 * d, t=t, std=std)
    rate = torch.rand(d, generator=g, device="cuda") ** 3 * fast + 1e-4
    params = torch.stack([rate, randn(g, d, std=0.5), randn(g, d, std=0.5)])
    return g, P, params


def gates(P, params):
    """fall, a, i, s and v in float64."""
    d = params.shape[1]
    rate, b_a, b_i = params.to(F64)
    P = P.to(F64)
    fall = rate * torch.sigmoid(P[..., :d] + b_a)
    i = torch.sigmoid(P[..., d:2 * d] + b_i)
    return fall, torch.exp(-fall), i, torch.sqrt(-torch.expm1(-2 * fall)), P[..., 2 * d:]


def spans(B, T, cu):
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    return [(0, int(s), int(e)) for s, e in zip(cu[:-1], cu[1:])]


def reference(P, params, cu=None, state=None):
    """(H, last, bounds of their errors) by a float64 unroll."""
    B, T, d = P.shape[0], P.shape[1], P.shape[2] // 3
    fall, a, i, s, v = (x.cpu() for x in gates(P, params))
    u = s * i * v
    c = (4 + 2 * fall) * 2.0 ** -21
    H, E = torch.zeros(B, T, d, dtype=F64), torch.zeros(B, T, d, dtype=F64)
    seqs = spans(B, T, cu)
    last, e_last = torch.zeros(len(seqs), d, dtype=F64), torch.zeros(len(seqs), d, dtype=F64)
    for r, (b, t0, t1) in enumerate(seqs):
        h = torch.zeros(d, dtype=F64) if state is None else state[r].cpu().to(F64)
        e = torch.zeros(d, dtype=F64)
        for t in range(t0, t1):
            ah = a[b, t] * h
            e = a[b, t] * e + c[b, t] * (ah.abs() + u[b, t].abs())
            h = ah + u[b, t]
            H[b, t], E[b, t] = h, e
        last[r], e_last[r] = h, e
    return H.cuda(), last.cuda(), E.cuda(), e_last.cuda()


def reference_backward(P, params, H, gH, cu=None, state=None, g_last=None):
    B, T, d = P.shape[0], P.shape[1], P.shape[2] // 3
    fall, a, i, s, v = (x.cpu() for x in gates(P, params))
    rate = params[0].to(F64).cpu()
    r = fall / rate
    omr, omi = torch.sigmoid(-(P[..., :d].to(F64) + params[1].to(F64))).cpu(), torch.sigmoid(-(P[..., d:2 * d].to(F64) + params[2].to(F64))).cpu()
    c = (4 + 2 * fall) * 2.0 ** -21
    H, gH = H.to(F64).cpu(), gH.to(F64).cpu()
    before = torch.zeros_like(H)
    G, E = torch.zeros_like(H), torch.zeros_like(H)
    seqs = spans(B, T, cu)
    g0, e0 = torch.zeros(len(seqs), d, dtype=F64), torch.zeros(len(seqs), d, dtype=F64)
    for k, (b, t0, t1) in enumerate(seqs):
        nu = torch.zeros(d, dtype=F64) if g_last is None else g_last[k].cpu().to(F64)
        e = torch.zeros(d, dtype=F64)
        for t in range(t1 - 1, t0 - 1, -1):
            before[b, t] = H[b, t - 1] if t > t0 else 0.0 if state is None else state[k].cpu().to(F64)
            G[b, t] = gH[b, t] + nu
            E[b, t] = e + c[b, t] * (gH[b, t].abs() + nu.abs())
            e = a[b, t] * E[b, t] + c[b, t] * (a[b, t] * G[b, t]).abs()
            nu = a[b, t] * G[b, t]
        g0[k], e0[k] = nu, e
    over = a * a / s
    w, scale = G * (a * before - over * i * v), (a * before).abs() + (over * i * v).abs()
    dw = (E + 4 * c * G.abs()) * scale
    g_a, d_a = -w * rate * r * omr, (dw + 4 * c * w.abs()) * rate * r * omr
    g_i, d_i = G * s * v * i * omi, (E + 4 * c * G.abs()) * (s * v * i * omi).abs()
    g_v, d_v = G * s * i, (E + 4 * c * G.abs()) * s * i
    sums = torch.stack([-(w * r).sum((0, 1)), g_a.sum((0, 1)), g_i.sum((0, 1))])
    mags = torch.stack([(w * r).abs().sum((0, 1)), g_a.abs().sum((0, 1)), g_i.abs().sum((0, 1))])
    offs = torch.stack([((dw + 4 * c * w.abs()) * r).sum((0, 1)), d_a.sum((0, 1)), d_i.sum((0, 1))])
    offs = offs + mags * (B * T) * 2.0 ** -24       # sums of B T terms in any order
    return (torch.cat([g_a, g_i, g_v], -1).cuda(), torch.cat([d_a, d_i, d_v], -1).cuda(), sums.cuda(), offs.cuda(),
            g0.cuda(), e0.cuda())


SHAPES = [(1, 1, 8), (2, 2, 40), (3, 63, 32), (1, 64, 72), (2, 65, 264), (1, 300, 136), (5, 129, 64), (1, 2500, 64), (40, 70, 8),
          (70, 300, 8), (130, 300, 8), (6, 700, 1408), (66, 64, 72), (260, 260, 8)]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("B,T,d", SHAPES)
def test_forward_and_backward(B, T, d, given, t):
    g, P, params = inputs(B, T, d, t, seed=B * T + d)
    state = randn(g, B, d) if given else None
    H, last = nr.linear_recurrence(P, params, state=state)
    ref, ref_last, E, e_last = reference(P, params, state=state)
    check(H, ref, E + rounding(t) * ref.abs(), "H")
    check(last, ref_last, e_last, "last")
    gH = randn(g, B, T, d, t=t)
    g_last = randn(g, B, d) if given else None
    r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=g_last)
    gP, dP, sums, offs, g0, e0 = reference_backward(P, params, H, gH, state=state, g_last=g_last)
    check(r.gP, gP, dP + rounding(t) * gP.abs(), "gP")
    check(r.gparams, sums, offs, "gparams")
    if given:
        check(r.g_state, g0, e0, "g_state")
    else:
        assert r.g_state is None


PACKS = [[0, 1], [0, 0, 5, 5, 6, 70, 70], [0, 64, 128, 192], [0, 63, 64, 129, 129, 400], [0, 1000, 1001, 1300],
         list(range(0, 190)), [0, 7, 900, 900]]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("pack", range(len(PACKS)))
def test_packs(pack, given, t):
    packs_of_width(pack, 40, given, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("pack", [1, 3, 5, 6])
def test_wide_packs(pack, t):
    """More than 128 tiles of units: the form with copies a tile ahead."""
    packs_of_width(pack, 8216, True, t)


LONG_PACKS = [[0, 300, 1100, 1100, 1101, 2400, 2433, 4100], [0, 64, 2048, 2048, 2112, 4096], [0, 0, 1, 1500, 3000, 3000]]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("pack", range(len(LONG_PACKS)))
def test_packs_cut_by_segments(pack, given, t):
    """Segments enough and long enough to be columns of their own: 64-unit tiles times
    segments from 128 on (fp32 forward 256), and eight chunks a segment on average."""
    packs_of_width(LONG_PACKS[pack], 1800 if t == torch.bfloat16 else 3400, given, t)


def test_short_chunks_leave_the_next_segment_alone():
    """What a segment's short last chunk loads beyond its end, NaN and infinities, reaches
    nothing, and nothing is written there by it."""
    cu, d = [0, 700, 1419, 2200, 4000], 2056
    N = cu[-1]
    g, P, params = inputs(1, N, d, torch.bfloat16, seed=21)
    gH = randn(g, 1, N, d, t=torch.bfloat16)
    H, last = nr.linear_recurrence(P, params, cu_seqlens=cu)
    r = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=cu)
    Q, gQ, HQ = P.clone(), gH.clone(), H.clone()
    for x, bad in ((Q, float("nan")), (gQ, float("inf")), (HQ, float("nan"))):
        x[0, 1419:2200] = bad
    H2, last2 = nr.linear_recurrence(Q, params, cu_seqlens=cu)
    r2 = nr.linear_recurrence_backward(Q, params, HQ, gQ, cu_seqlens=cu)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[1419:2200] = False
    assert torch.equal(H2[0, keep], H[0, keep]) and torch.equal(r2.gP[0, keep], r.gP[0, keep])
    assert torch.equal(last2[[0, 1, 3]], last[[0, 1, 3]])
    again = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=cu)
    assert all(torch.equal(x, y) for x, y in zip(r[:2], again[:2]))


def packs_of_width(pack, d, given, t):
    bounds = PACKS[pack] if isinstance(pack, int) else pack
    cu = torch.tensor(bounds, dtype=torch.int32)
    N, S = bounds[-1], len(bounds) - 1
    g, P, params = inputs(1, N, d, t, seed=len(bounds))
    state = randn(g, S, d) if given else None
    H, last = nr.linear_recurrence(P, params, cu_seqlens=cu, state=state)
    ref, ref_last, E, e_last = reference(P, params, bounds, state)
    check(H, ref, E + rounding(t) * ref.abs(), "H")
    check(last, ref_last, e_last, "last")
    gH, g_last = randn(g, 1, N, d, t=t), randn(g, S, d) if given else None
    r = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=nr.DeviceCuSeqlens(cu, N, "cuda:0"), state=state, g_state=g_last)
    gP, dP, sums, offs, g0, e0 = reference_backward(P, params, H, gH, bounds, state, g_last)
    check(r.gP, gP, dP + rounding(t) * gP.abs(), "gP")
    check(r.gparams, sums, offs, "gparams")
    if given:
        check(r.g_state, g0, e0, "g_state")


def test_gradients_against_differences():
    """d/dtheta of sum(gH H) + sum(g_last last) by central differences of the float64 unroll."""
    B, T, d = 2, 9, 8
    g, P, params = inputs(B, T, d, torch.float32, seed=3)
    state, gH, g_last = randn(g, B, d), randn(g, B, T, d), randn(g, B, d)
    H, _ = nr.linear_recurrence(P, params, state=state)
    r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=g_last)

    def value(p, w, s):
        fall, a, i, q, v = gates(p, w)
        h, total = s, 0.0
        for t in range(T):
            h = a[:, t] * h + (q * i * v)[:, t]
            total = total + (gH[:, t].to(F64) * h).sum()
        return total + (g_last.to(F64) * h).sum()
    step = 1e-5
    at = [P.to(F64), params.to(F64), state.to(F64)]
    for which, got in ((0, r.gP), (1, r.gparams), (2, r.g_state)):
        for n in torch.randint(0, at[which].numel(), (12,), generator=g, device="cuda").tolist():
            pair = []
            for sign in (1, -1):
                moved = [x.clone() for x in at]
                moved[which].view(-1)[n] += sign * step
                pair.append(value(*moved))
            slope = float((pair[0] - pair[1]) / (2 * step))
            # differences: 1e-8 of the values' size and step^2 of the third derivative (1/rate^2.5 for a rate)
            tiny = float(at[1][0, n]) if which == 1 and n < d else 1.0
            tol = 2e-5 * (1 + abs(slope)) if tiny > 0.01 else None
            if tol is not None:
                assert abs(float(got.view(-1)[n]) - slope) <= tol, (which, n)


@pytest.mark.parametrize("t", TYPES)
def test_steps_follow_the_forward(t):
    """Prefill, then one step after another, against one forward over all of it."""
    B, T, d, more = 5, 130, 72, 6
    g, P, params = inputs(B, T + more, d, t, seed=9)
    ref, ref_last, E, e_last = reference(P, params)
    H, state = nr.linear_recurrence(P[:, :T], params)
    check(H, ref[:, :T], E[:, :T] + rounding(t) * ref[:, :T].abs())
    for j in range(T, T + more):
        h, new = nr.linear_recurrence_step(params, state, P[:, j])
        check(h, ref[:, j], E[:, j] + rounding(t) * ref[:, j].abs())
        again = state.clone()
        nr.linear_recurrence_step(params, again, P[:, j], state_out=again)     # in place
        assert torch.equal(again, new)
        state = new
    check(state, ref_last, e_last)
    h0, s0 = nr.linear_recurrence_step({k: v for k, v in zip(nr.RECURRENCE_ORDER, params)}, None, P[:, 0])
    check(s0, ref[:, 0], E[:, 0])
    # a forward that continues from a state
    H1, s1 = nr.linear_recurrence(P[:, :70], params)
    H2, s2 = nr.linear_recurrence(P[:, 70:], params, state=s1)
    check(torch.cat([H1, H2], 1), ref, E + rounding(t) * ref.abs())
    check(s2, ref_last, e_last)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("slots,d", [(1, 8), (3, 40), (257, 264), (1000, 1024)])
def test_step_sizes(slots, d, t):
    g, P, params = inputs(slots, 1, d, t, seed=slots)
    state = randn(g, slots, d)
    h, s = nr.linear_recurrence_step(params, state, P[:, 0])
    fall, a, i, q, v = gates(P[:, 0], params)
    ref = a * state.to(F64) + q * i * v
    tol = (4 + 2 * fall) * 2.0 ** -21 * ((a * state).abs() + (q * i * v).abs())
    check(s, ref, tol)
    check(h, ref, tol + rounding(t) * ref.abs())


def test_extreme_gates():
    """Gates that are open or shut to the last bit, rates of zero and large, give finite values and gradients."""
    d, T = 16, 40
    P = torch.zeros(1, T, 3 * d, device="cuda")
    big = torch.tensor([-3e38, -200.0, -90.0, 90.0, 200.0, 3e38, 0.0, -30.0], device="cuda")
    P[..., :d] = big.repeat(2)
    P[..., d:2 * d] = big.flip(0).repeat_interleave(2)
    P[..., 2 * d:] = 1.0
    rate = torch.tensor([0.0, 1e-30, 1e-6, 1.0, 50.0, 1e4, 0.5, 0.1], device="cuda").repeat_interleave(2)
    params = torch.stack([rate, torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    state = torch.ones(1, d, device="cuda")
    H, last = nr.linear_recurrence(P, params, state=state)
    assert bool(H.isfinite().all())
    ref, ref_last, E, e_last = reference(P, params, state=state)
    # a sigmoid is bounded below by 2^-63: s by 2^-31 sqrt(2 rate), over T steps
    floor = T * 2.0 ** -31 * (2 * rate.to(F64)).sqrt() * 1.01
    check(H, ref, E + floor)
    gH = torch.ones(1, T, d, device="cuda")
    r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=state)
    for x in r:
        assert bool(x.isfinite().all())


def test_a_bad_value_stays_in_its_unit_and_sequence():
    B, T, d = 3, 200, 40
    g, P, params = inputs(B, T, d, torch.float32, seed=4)
    clean, _ = nr.linear_recurrence(P, params)
    for bad in (float("nan"), float("inf"), -float("inf")):
        Q = P.clone()
        Q[1, 77, 2 * d + 5] = bad
        H, last = nr.linear_recurrence(Q, params)
        hit = torch.zeros(B, T, d, dtype=torch.bool, device="cuda")
        hit[1, 77:, 5] = True
        assert torch.equal(H[~hit], clean[~hit])
        assert not bool(H[hit][:1].isfinite().any())
    # in a pack nothing crosses a segment's bounds, in either direction
    cu = torch.tensor([0, 90, 110, 200], dtype=torch.int32)
    gH = randn(g, 1, T, d)
    Q = P[:1].clone()
    H0, l0 = nr.linear_recurrence(Q, params, cu_seqlens=cu)
    r0 = nr.linear_recurrence_backward(Q, params, H0, gH, cu_seqlens=cu)
    Q[0, 90:110], gH1 = float("nan"), gH.clone()
    gH1[0, 90:110] = float("inf")
    H, last = nr.linear_recurrence(Q, params, cu_seqlens=cu)
    r = nr.linear_recurrence_backward(Q, params, H, gH1, cu_seqlens=cu)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[90:110] = False
    assert torch.equal(H[0, keep], H0[0, keep]) and torch.equal(last[[0, 2]], l0[[0, 2]])
    assert torch.equal(r.gP[0, keep], r0.gP[0, keep])


def test_empty_inputs():
    d = 16
    g, P, params = inputs(2, 1, d, torch.float32)
    state = randn(g, 2, d)
    H, last = nr.linear_recurrence(P[:, :0], params, state=state)
    assert H.shape == (2, 0, d) and torch.equal(last, state)
    assert torch.equal(nr.linear_recurrence(P[:, :0], params)[1], torch.zeros(2, d, device="cuda"))
    r = nr.linear_recurrence_backward(P[:, :0], params, H, H, state=state, g_state=state)
    assert torch.equal(r.g_state, state) and torch.equal(r.gparams, torch.zeros(3, d, device="cuda"))
    H, last = nr.linear_recurrence(P[:0], params)
    assert H.shape == (0, 1, d) and last.shape == (0, d)
    r = nr.linear_recurrence_backward(P[:0], params, H, H)
    assert torch.equal(r.gparams, torch.zeros(3, d, device="cuda"))
    h, s = nr.linear_recurrence_step(params, None, P[:0, 0])
    assert h.shape == (0, d)


@pytest.mark.parametrize("t", TYPES)
def test_repeats_strides_streams_and_outputs(t):
    B, T, d = 3, 1000, 264
    g, P, params = inputs(B, T, d, t, seed=11)
    state, gH = randn(g, B, d), randn(g, B, T, d, t=t)
    H, last = nr.linear_recurrence(P, params, state=state)
    r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=last)
    for _ in range(3):                              # nothing depends on the order of threads
        H2, last2 = nr.linear_recurrence(P, params, state=state)
        r2 = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=last)
        assert torch.equal(H, H2) and torch.equal(last, last2)
        assert all(torch.equal(x, y) for x, y in zip(r, r2))
    wide = torch.empty(B, T, 3 * d + 8, dtype=t, device="cuda")
    wide[..., :3 * d] = P
    assert torch.equal(nr.linear_recurrence(wide[..., :3 * d], params, state=state)[0], H)   # strided: copied
    out = torch.empty_like(H)
    assert nr.linear_recurrence(P, params, state=state, out=out)[0] is out and torch.equal(out, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        H3, _ = nr.linear_recurrence(P, params, state=state)
        r3 = nr.linear_recurrence_backward(P, params, H3, gH, state=state, g_state=last)
    H4, _ = nr.linear_recurrence(P, params, state=state)      # at the same time, on this stream
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(H3, H) and torch.equal(H4, H) and all(torch.equal(x, y) for x, y in zip(r, r3))


@pytest.mark.parametrize("t", TYPES)
def test_captured_and_replayed(t):
    B, T, d = 2, 500, 72
    g, P, params = inputs(B, T, d, t, seed=12)
    state, gH = randn(g, B, d), randn(g, B, T, d, t=t)
    nr.linear_recurrence(P, params, state=state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H, last = nr.linear_recurrence(P, params, state=state)
        r = nr.linear_recurrence_backward(P, params, H, gH, state=state, g_state=last)
        h, s = nr.linear_recurrence_step(params, last, P[:, 0])
    for seed in (13, 14):
        _, Q, _ = inputs(B, T, d, t, seed=seed)
        P.copy_(Q)
        graph.replay()
        H2, last2 = nr.linear_recurrence(Q, params, state=state)
        r2 = nr.linear_recurrence_backward(Q, params, H2, gH, state=state, g_state=last2)
        assert torch.equal(H, H2) and torch.equal(last, last2) and all(torch.equal(x, y) for x, y in zip(r, r2))
        assert torch.equal(s, nr.linear_recurrence_step(params, last2, Q[:, 0])[1])


def test_refusals():
    g, P, params = inputs(2, 4, 16, torch.float32)
    H = torch.zeros(2, 4, 16, device="cuda")
    for call in (lambda: nr.linear_recurrence(P.cpu(), params),
                 lambda: nr.linear_recurrence(P[0], params),
                 lambda: nr.linear_recurrence(P, params[:2]),
                 lambda: nr.linear_recurrence(P, params, state=H[0]),
                 lambda: nr.linear_recurrence(P, params, state=torch.zeros(2, 16, dtype=torch.float64, device="cuda")),
                 lambda: nr.linear_recurrence(P, params, cu_seqlens=[0, 4]),
                 lambda: nr.linear_recurrence(P, params, out=H[:, ::2]),
                 lambda: nr.linear_recurrence(P, params, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
                 lambda: nr.linear_recurrence_backward(P, params, H[:1], H),
                 lambda: nr.linear_recurrence_backward(P, params, H, H.bfloat16()),
                 lambda: nr.linear_recurrence_step(params, H[:, 0].double(), P[:, 0]),
                 lambda: nr.linear_recurrence_step(params, None, P[:, 0], state_out=H[:, 0]),
                 lambda: nr.linear_recurrence_step(params, None, P)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: nr.linear_recurrence(P.double(), params), lambda: nr.linear_recurrence(P[..., :36], params[:, :12])):
        with pytest.raises(TypeError):
            call()


def test_offsets_beyond_32_bits():
    """The last steps of more than 2^32 preactivations against a call over them alone.

    Decays are at most exp(-0.5 sig(-2.7)) < 0.97, so that 0.97^2000 < 2^-80 of what came
    before is left.  Two scans of the same steps in other groups differ by at most their
    errors: (4 + 2 fall) 2^-21 of magnitudes below 32, 33 times over (1 / (1 - 0.97)),
    with fall <= 1: 33 * 32 * 6 * 2^-21 < 2^-8 each, and a result's rounding."""
    T, d, n = 1400003, 1024, 4000
    g = gen(7)
    P = torch.empty(1, T, 3 * d, dtype=torch.bfloat16, device="cuda").uniform_(-2.5, 2.5, generator=g)
    assert P.numel() > 1 << 32
    params = torch.stack([torch.rand(d, generator=g, device="cuda") / 2 + 0.5, randn(g, d, std=0.05).clamp(-0.2, 0.2),
                          torch.zeros(d, device="cuda")])

    def same(got, want):
        got, want = got.to(F64), want.to(F64)
        return bool(((got - want).abs() <= 2.0 ** -8 * (got.abs() + want.abs()) + 2.0 ** -7).all()) and \
            bool(want.abs().max() < 32) and bool(want.abs().max() > 0.5)
    H, last = nr.linear_recurrence(P, params)
    tail = P[:, -n:].contiguous()
    H_tail, last_tail = nr.linear_recurrence(tail, params)
    assert same(H[:, -n // 2:], H_tail[:, -n // 2:]) and same(last, last_tail)
    gH = torch.empty(1, T, d, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1, generator=g)
    gP = nr.linear_recurrence_backward(P, params, H, gH).gP
    gP_tail = nr.linear_recurrence_backward(tail, params, H[:, -n:].contiguous(), gH[:, -n:].contiguous(),
                                            state=H[:, -n - 1].float().contiguous()).gP
    assert same(gP[:, -n // 2:], gP_tail[:, -n // 2:])
