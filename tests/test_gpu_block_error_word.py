"""The error word of the recurrence's workspace after calls without work: a caller that polls
it must not read what was there before as a wait that gave up."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


def error_word(ws):
    return ws[:8].view(torch.int32).tolist()[1]


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T", [(2, 0), (0, 5), (0, 0), (2, 5)])
def test_recurrence(B, T, t):
    d = 16
    params = torch.stack([torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    P, H = torch.ones(B, T, 3 * d, dtype=t, device="cuda"), torch.zeros(B, T, d, dtype=t, device="cuda")
    for state in (None, torch.ones(B, d, device="cuda")):
        ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        _, last = nr.linear_recurrence(P, params, state=state, workspace=ws)
        assert error_word(ws) == 0
        if T == 0:
            assert torch.equal(last, torch.zeros(B, d, device="cuda") if state is None else state)
        ws.fill_(255)
        r = nr.linear_recurrence_backward(P, params, H, H, state=state, g_state=state, workspace=ws)
        assert error_word(ws) == 0
        if B * T == 0:
            assert not bool(r.gparams.any())


@pytest.mark.parametrize("cu", [[0, 0], [0, 0, 0, 0]])
def test_a_pack_without_steps(cu):
    d = 16
    params = torch.stack([torch.ones(d, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    P, H, state = torch.ones(1, 0, 3 * d, device="cuda"), torch.zeros(1, 0, d, device="cuda"), torch.randn(len(cu) - 1, d, device="cuda")
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    _, last = nr.linear_recurrence(P, params, cu_seqlens=cu, state=state, workspace=ws)
    assert error_word(ws) == 0 and torch.equal(last, state)
    ws.fill_(255)
    r = nr.linear_recurrence_backward(P, params, H, H, cu_seqlens=cu, state=state, g_state=state, workspace=ws)
    assert error_word(ws) == 0 and torch.equal(r.g_state, state) and not bool(r.gparams.any())


def test_a_feed_forward_of_no_rows_leaves_its_workspace_alone():
    W_in, W_out = torch.ones(48, 16, device="cuda"), torch.ones(16, 24, device="cuda")
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    nr.gated_mlp(torch.ones(0, 16, device="cuda"), W_in, W_out, workspace=ws)
    assert bool((ws == 255).all())
