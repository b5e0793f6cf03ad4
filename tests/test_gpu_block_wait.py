"""Waits that give up in the recurrence and the feed-forward block: the call ends, sets
its workspace's error word, and leaves NaN where the wait mattered; the next call with
the usual limit is unharmed."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


def randn(seed, *shape, t=torch.float32, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(t)


def words(ws):
    return ws[:8].view(torch.int32).tolist()


@pytest.fixture
def short_waits():
    def limit(ns):
        old.append(nr.set_wait_limit_ns(ns))
    old = []
    yield limit
    nr.set_wait_limit_ns(2_000_000_000)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_recurrence(t, short_waits):
    B, T, d = 2, 20000, 64
    P = randn(1, B, T, 3 * d, t=t)
    params = torch.stack([torch.full((d,), 0.1, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    gH = randn(2, B, T, d, t=t)
    H, last = nr.linear_recurrence(P, params)
    r = nr.linear_recurrence_backward(P, params, H, gH)
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    short_waits(1)
    H1, last1 = nr.linear_recurrence(P, params, workspace=ws)
    torch.cuda.synchronize()
    gave_up = words(ws)[1] != 0
    # what did not wait, or waited successfully, is right; the rest is NaN
    same = (H1 == H) | H1.isnan()
    assert bool(same.all()) and (gave_up or torch.equal(H1, H))
    assert gave_up and bool(H1.isnan().any())
    r1 = nr.linear_recurrence_backward(P, params, H, gH, workspace=ws)
    torch.cuda.synchronize()
    assert words(ws)[1] != 0 and bool(r1.gP.isnan().any())
    assert bool(((r1.gP == r.gP) | r1.gP.isnan()).all())
    nr.set_wait_limit_ns(2_000_000_000)
    H2, last2 = nr.linear_recurrence(P, params, workspace=ws)
    torch.cuda.synchronize()
    assert words(ws)[1] == 0 and torch.equal(H2, H) and torch.equal(last2, last)
    r2 = nr.linear_recurrence_backward(P, params, H, gH, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(r[:2], r2[:2]))


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_gated_mlp(t, short_waits):
    n, d, f = 3000, 256, 520
    x, W_in, W_out, g = randn(1, n, d, t=t), randn(2, 2 * f, d, t=t, std=0.06), randn(3, d, f, t=t, std=0.04), randn(4, n, d, t=t)
    y, kept = nr.gated_mlp(x, W_in, W_out, keep=True)
    r = nr.gated_mlp_backward(x, W_in, W_out, kept, g)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for limit in (1, 300, 3000, 30000):
        short_waits(limit)
        y1, kept1 = nr.gated_mlp(x, W_in, W_out, keep=True, workspace=ws)
        torch.cuda.synchronize()
        assert bool(((y1 == y) | y1.isnan()).all())
        if limit == 1:
            assert words(ws)[0] != 0 and bool(y1.isnan().any())
        r1 = nr.gated_mlp_backward(x, W_in, W_out, kept, g, workspace=ws)
        torch.cuda.synchronize()
        for p, q in zip(r1, r):
            assert bool(((p == q) | p.isnan()).all())
        if limit == 1:
            assert words(ws)[0] != 0 and all(bool(p.isnan().any()) for p in r1)
        nr.set_wait_limit_ns(2_000_000_000)
        y2, kept2 = nr.gated_mlp(x, W_in, W_out, keep=True, workspace=ws)
        r2 = nr.gated_mlp_backward(x, W_in, W_out, kept2, g, workspace=ws)
        torch.cuda.synchronize()
        assert words(ws)[0] == 0 and torch.equal(y2, y) and all(torch.equal(p, q) for p, q in zip(r2, r))
