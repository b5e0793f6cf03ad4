"""Packs of the gated linear recurrence that go by their segments and packs of as many segments
of which one is too long for that: both ways and their border, against a float64 unroll.

By segments: unit tiles (of 64) times segments from 128 on (fp32 forward 256), eight chunks a
segment on average (a chunk: 32 steps in fp32, 64 in bf16), and the longest segment's chunks
at most a hundredth (backward: 140th) of all chunks times unit tiles."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr
from test_gpu_linear_recurrence import TYPES, check, inputs, packs_of_width, randn, reference, reference_backward, rounding

pytestmark = pytest.mark.gpu

#: of 5100 to 5300 steps; bf16, whose chunks are twice as long: of twice as many
EVEN = [0, 520, 1, 512, 513, 575, 64, 600, 448, 449, 33, 577, 0, 520, 388]
LENGTHS = {"even": EVEN, "even, empty ends": [0, 0, *[523] * 10, 0], "one long": [31, 64, 0, 1, 65, 33, 2, 4900, 64, 63, 7, 1],
           "one long first": [4600, 1, 64, 65, 0, 100, 128, 129, 40, 1, 1], "one long last": [100, 64, 0, 65, 128, 129, 40, 33, 1, 4700],
           "two": [2600, 0, 0, 1, 0, 0, 0, 2601, 0]}


def offsets(lengths, t=torch.float32):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n * (2 if t == torch.bfloat16 else 1))
    return cu


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("name", LENGTHS)
def test_against_the_unroll(name, given, t):
    packs_of_width(offsets(LENGTHS[name], t), 1864, given, t)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("longest", range(3))
def test_beside_the_border(longest, t):
    """Fifteen segments over 18 unit tiles: the longest of them just by segments, just not in
    the backward, just not in the forward."""
    L, tiles, S = (64 if t == torch.bfloat16 else 32), 18, 15
    rest = 9                                          # chunks of the others
    most = [next(c for c in range(1000) if (c + 1) * k > (c + 1 + rest * (S - 1)) * tiles) for k in (140, 100)]
    chunks = (most[0], most[0] + 1, most[1] + 1)[longest]
    packs_of_width(offsets([rest * L] * 7 + [chunks * L] + [rest * L] * 7), tiles * 64, True, t)


@pytest.mark.parametrize("name", ["even", "one long"])
def test_a_bad_segment_stays_alone(name):
    """What a segment's short last chunk loads beyond its end, NaN and infinities, reaches
    nothing, and nothing is written there by it."""
    cu, d = offsets(LENGTHS[name], torch.bfloat16), 1864
    N, bad = cu[-1], 4                                # a segment of 1026 or 130 steps
    g, P, params = inputs(1, N, d, torch.bfloat16, seed=21)
    gH = randn(g, 1, N, d, t=torch.bfloat16)
    H, last = nr.linear_recurrence(P, params, cu_seqlens=cu)
    r = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=cu)
    Q, gQ, HQ = P.clone(), gH.clone(), H.clone()
    for x, v in ((Q, float("nan")), (gQ, float("inf")), (HQ, float("nan"))):
        x[0, cu[bad]:cu[bad + 1]] = v
    H2, last2 = nr.linear_recurrence(Q, params, cu_seqlens=cu)
    r2 = nr.linear_recurrence_backward(Q, params, HQ, gQ, cu_seqlens=cu)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[cu[bad]:cu[bad + 1]] = False
    assert torch.equal(H2[0, keep], H[0, keep]) and torch.equal(r2.gP[0, keep], r.gP[0, keep])
    live = [k for k in range(len(cu) - 1) if k != bad]
    assert torch.equal(last2[live], last[live])


@pytest.mark.parametrize("t", TYPES)
def test_one_captured_call_for_packs_of_either_kind(t):
    """The way is chosen when the call runs: a captured call whose offsets change in place."""
    d, S = 1864, 12
    kinds = [offsets([433] * 11 + [437], t), offsets([31, 64, 0, 1, 65, 33, 2, 4900, 64, 33, 6, 1], t)]
    N = kinds[0][-1]
    assert kinds[1][-1] == N
    g, P, params = inputs(1, N, d, t, seed=5)
    state, gH = randn(g, S, d), randn(g, 1, N, d, t=t)
    pack = nr.DeviceCuSeqlens(torch.tensor(kinds[0], dtype=torch.int32), N)
    nr.linear_recurrence(P, params, cu_seqlens=pack, state=state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        H, last = nr.linear_recurrence(P, params, cu_seqlens=pack, state=state)
        r = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=pack, state=state, g_state=last)
    for kind in (*kinds, *kinds):
        pack.tensor.copy_(torch.tensor(kind, dtype=torch.int32))
        graph.replay()
        ref, ref_last, E, e_last = reference(P, params, kind, state)
        check(H, ref, E + rounding(t) * ref.abs(), "H")
        check(last, ref_last, e_last, "last")
        gP, dP, sums, offs, g0, e0 = reference_backward(P, params, H, gH, kind, state, last)
        check(r.gP, gP, dP + rounding(t) * gP.abs(), "gP")
        check(r.gparams, sums, offs, "gparams")
        check(r.g_state, g0, e0, "g_state")
        again = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=kind, state=state, g_state=last)
        assert all(torch.equal(x, y) for x, y in zip(r, again))
