"""Waits that give up in the recurrence over packs, by their segments and by the time axis: the
call ends and sets its error word, what it gives is right or NaN, and the next call with the
usual limit is unharmed."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lengths", [[1640] * 40, [20] * 20 + [64800] + [20] * 20])
def test_packs(lengths, t):
    d = 512
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    N = cu[-1]
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    P = torch.randn(1, N, 3 * d, generator=g, device="cuda").to(t)
    gH = torch.randn(1, N, d, generator=g, device="cuda").to(t)
    params = torch.stack([torch.full((d,), 0.1, device="cuda"), torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda")])
    pack = nr.DeviceCuSeqlens(torch.tensor(cu, dtype=torch.int32), N)
    H, last = nr.linear_recurrence(P, params, cu_seqlens=pack)
    r = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=pack)
    ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def word():
        return ws[:8].view(torch.int32).tolist()[1]
    try:
        nr.set_wait_limit_ns(1)
        H1, _ = nr.linear_recurrence(P, params, cu_seqlens=pack, workspace=ws)
        assert word() != 0 and bool(H1.isnan().any()) and bool(((H1 == H) | H1.isnan()).all())
        r1 = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=pack, workspace=ws)
        assert word() != 0 and bool(r1.gP.isnan().any()) and bool(((r1.gP == r.gP) | r1.gP.isnan()).all())
    finally:
        nr.set_wait_limit_ns(2_000_000_000)
    H2, last2 = nr.linear_recurrence(P, params, cu_seqlens=pack, workspace=ws)
    assert word() == 0 and torch.equal(H2, H) and torch.equal(last2, last)
    r2 = nr.linear_recurrence_backward(P, params, H, gH, cu_seqlens=pack, workspace=ws)
    assert word() == 0 and all(torch.equal(x, y) for x, y in zip(r[:2], r2[:2]))
