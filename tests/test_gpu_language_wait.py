"""Bounded waits of the vocabulary loss that run out: the call ends, its error word
and NaN tell, and the next call is right."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


def error_word(ws):
    return int(ws[4:8].view(torch.int32))


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,V,d", [(40, 3000, 96), (300, 5000, 515), (3000, 9000, 1024)])
def test_a_wait_that_runs_out_is_reported(n, V, d, t):
    """No accumulator is there within a nanosecond of the launch, so the epilogues'
    first waits run out, with copies and products of both CTAs of a pair in flight."""
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    x, W = (torch.randn(*s, d, generator=g, device="cuda").to(t) for s in ((n,), (V,)))
    at = torch.randint(0, V, (n,), generator=g, device="cuda")
    gl = torch.ones(n, device="cuda")
    ws = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    loss, lse = nr.vocab_loss(x, W, at, workspace=ws)
    assert error_word(ws) == 0
    grads = nr.vocab_loss_backward(x, W, at, lse, gl, workspace=ws)
    assert error_word(ws) == 0
    limit = nr.set_wait_limit_ns(1)
    try:
        for _ in range(3):
            late = nr.vocab_loss(x, W, at, workspace=ws)
            assert error_word(ws) != 0
            assert bool(late[0].isnan().any()) and bool(late[1].isnan().any())
            late = nr.vocab_loss_backward(x, W, at, lse, gl, workspace=ws)
            assert error_word(ws) != 0
            assert bool(late[0].isnan().any()) and bool(late[1].isnan().any())
    finally:
        assert nr.set_wait_limit_ns(limit) == 1
    again = nr.vocab_loss(x, W, at, workspace=ws)
    assert error_word(ws) == 0
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
    again = nr.vocab_loss_backward(x, W, at, lse, gl, workspace=ws)
    assert error_word(ws) == 0
    assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
def test_what_is_not_nan_after_a_wait_ran_out_is_right(t):
    """Limits about as long as the waits are: some pairs give up, at different places.
    An output that is a number is the one that the call gives with time enough."""
    n, V, d = 900, 12000, 515
    g = torch.Generator(device="cuda")
    g.manual_seed(32)
    x, W = (torch.randn(*s, d, generator=g, device="cuda").to(t) for s in ((n,), (V,)))
    at = torch.randint(0, V, (n,), generator=g, device="cuda")
    gl = torch.ones(n, device="cuda")
    ws = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    good = nr.vocab_loss(x, W, at, workspace=ws)
    good_grads = nr.vocab_loss_backward(x, W, at, good[1], gl, workspace=ws)
    old = nr.set_wait_limit_ns(1)
    try:
        for limit in (500, 1000, 2000, 3000, 5000, 8000, 12000, 20000, 50000):
            nr.set_wait_limit_ns(limit)
            for call, ref in ((lambda: nr.vocab_loss(x, W, at, workspace=ws), good),
                              (lambda: nr.vocab_loss_backward(x, W, at, good[1], gl, workspace=ws), good_grads)):
                for _ in range(3):
                    got = call()
                    gave_up = error_word(ws) != 0
                    for o, r in zip(got, ref):
                        same = o == r
                        assert bool((same | o.isnan()).all()) if gave_up else bool(same.all()), limit
    finally:
        nr.set_wait_limit_ns(old)
