"""Buffers that a caller hands in go to the kernels as addresses: what is not one
block of memory of the device they run on is refused before any launch."""
import pytest
import torch

import nonlinear_rnn_gb300 as nr
from nonlinear_rnn_gb300 import _binding, _language


def test_a_host_workspace_is_refused():
    host = torch.empty(4096, dtype=torch.uint8)
    for space in (_binding._space, _language._space):
        with pytest.raises(ValueError):
            space(host, 64, torch.device("cuda:0"))
        with pytest.raises(ValueError):
            space(host.numpy(), 64, torch.device("cuda:0"))


def calls():
    """Every call that takes a workspace or staging buffer, by name, at a small size."""
    t = dict(device="cuda")
    P, H = torch.zeros(1, 70, 96, **t), torch.zeros(1, 70, 32, **t)
    prm = torch.ones(6, 32)
    x, W, ids = torch.ones(5, 16, **t), torch.ones(48, 16, **t), torch.zeros(5, dtype=torch.int64, **t)
    lse = torch.zeros(5, **t)
    xb, Wb = torch.ones(1, 70, 32, dtype=torch.bfloat16, **t), torch.ones(96, 32, dtype=torch.bfloat16, **t)
    return {
        "newton_forward": lambda b: nr.newton_forward(P, prm, check=False, workspace=b),
        "newton_forward_x": lambda b: nr.newton_forward_x(xb, Wb, prm, check=False, workspace=b),
        "newton_backward": lambda b: nr.newton_backward(P, prm, H, H, workspace=b),
        "newton_forward_host": lambda b: nr.newton_forward_host(P.cpu(), prm, staging=b),
        "newton_forward_x_host": lambda b: nr.newton_forward_x_host(xb.cpu(), Wb, prm, staging=b, check=False),
        "input_projection": lambda b: nr.input_projection(x, W, workspace=b),
        "embedding_backward": lambda b: nr.embedding_backward(ids, x, 9, workspace=b),
        "block_norm_backward": lambda b: nr.block_norm_backward(x, g_u=x, workspace=b),
        "vocab_loss": lambda b: nr.vocab_loss(x, W, ids, workspace=b),
        "vocab_loss_backward": lambda b: nr.vocab_loss_backward(x, W, ids, lse, lse, workspace=b),
    }


@pytest.mark.gpu
def test_calls_refuse_buffers_that_are_not_theirs():
    room = 1 << 24
    for name, call in calls().items():
        for bad in (torch.empty(room, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(room),
                    torch.empty(2 * room, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(bad)
                pytest.fail(name)
        call(torch.empty(room, dtype=torch.uint8, device="cuda"))
        call(None)
    torch.cuda.synchronize()


def test_a_host_result_tensor_is_refused():
    with pytest.raises(ValueError):
        _binding._out(torch.empty(2, 3), (2, 3), torch.float32, torch.device("cuda:0"))


@pytest.mark.gpu
def test_calls_refuse_result_tensors_that_are_not_theirs():
    t = dict(device="cuda")
    P, prm = torch.zeros(1, 70, 96, **t), torch.ones(6, 32)
    x, W = torch.ones(5, 16, **t), torch.ones(48, 16, **t)
    xb, Wb = torch.ones(1, 70, 32, dtype=torch.bfloat16, **t), torch.ones(96, 32, dtype=torch.bfloat16, **t)
    f32, b16 = torch.float32, torch.bfloat16
    cases = {
        "newton_forward": (lambda o: nr.newton_forward(P, prm, check=False, out=o), (1, 70, 32), f32),
        "newton_forward_x": (lambda o: nr.newton_forward_x(xb, Wb, prm, check=False, out=o), (1, 70, 32), b16),
        "picard": (lambda o: nr.picard(P, prm, 2, out=o), (1, 70, 32), f32),
        "sequential_forward": (lambda o: nr.sequential_forward(P, prm, out=o), (1, 70, 32), f32),
        "decode_step": (lambda o: nr.decode_step(prm, preact=P[0, :5], out=o), (5, 32), f32),
        "input_projection": (lambda o: nr.input_projection(x, W, out=o), (5, 48), f32),
    }
    for name, (call, shape, dtype) in cases.items():
        numel = torch.Size(shape).numel()
        for bad in (torch.empty(shape, dtype=dtype), torch.empty(1, dtype=dtype, **t).expand(shape),
                    torch.empty(numel - 1, dtype=dtype, **t), torch.empty(shape, dtype=torch.float16, **t),
                    torch.empty(2 * numel, dtype=dtype, **t)[::2].view(shape)):
            with pytest.raises(ValueError):
                call(bad)
                pytest.fail(name)
        call(torch.empty(shape, dtype=dtype, **t))
    torch.cuda.synchronize()
