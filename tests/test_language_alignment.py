"""The fp32 vectors of the language-model operators (weights, their gradients, loss,
lse and dL/dloss) need four-byte alignment in either storage type: the C entry
points refuse others before any launch.  No GPU needed."""
import ctypes

import pytest

import nonlinear_rnn_gb300 as nr

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: the checks fail first
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("which", range(3))
def test_block_norm_weights(dtype, which):
    w = [FAKE] * 3
    w[which] = ODD
    assert nr.load().nrnn_block_norm_forward(FAKE, FAKE, FAKE, *w, dtype, 4, 16, 1e-6, FAKE, FAKE, None) == -1


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("which", range(6))
def test_block_norm_backward_weights_and_their_gradients(dtype, which):
    w = [FAKE] * 6
    w[which] = ODD
    # a workspace that is too small would be refused next (-7): no launch either way
    assert nr.load().nrnn_block_norm_backward(FAKE, FAKE, FAKE, *w[:3], FAKE, FAKE, dtype, 4, 16, 1e-6, FAKE, FAKE,
                                              FAKE, *w[3:], FAKE, 0, None) == -1


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("which", range(2))
@pytest.mark.parametrize("back", [0, 1])
def test_vocab_loss_vectors(dtype, which, back):
    v = [FAKE] * 2
    v[which] = ODD
    lib = nr.load()
    if back:
        st = lib.nrnn_vocab_loss_backward(FAKE, FAKE, dtype, 4, 16, 100, FAKE, 1, -100, 1.0, *v, FAKE, FAKE, FAKE, 0, None)
    else:
        st = lib.nrnn_vocab_loss_forward(FAKE, FAKE, dtype, 4, 16, 100, FAKE, 1, -100, 1.0, *v, FAKE, 0, None)
    assert st == -1
