"""Host-side checks of the language-model operators: workspace sizes and the
refusals, which come before any launch.  No GPU needed."""
import ctypes

import pytest
import torch

import nonlinear_rnn_gb300 as nr

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: the checks fail first
WS = ctypes.c_void_p(1 << 24)
BIG = 1 << 40


def test_embedding_refusals():
    f = nr.load().nrnn_embedding

    def call(ids=FAKE, kind=1, W=FAKE, dtype=1, n=4, V=10, d=16, out=FAKE):
        return f(ids, kind, W, dtype, n, V, d, -1, 1.0, out, None)
    assert call(n=0) == 0
    assert call(dtype=2) == -1
    assert call(kind=2) == -1
    assert call(n=-1) == -1
    assert call(V=0) == -1
    assert call(d=0) == -1
    assert call(ids=None) == -1
    assert call(W=None) == -1
    assert call(out=None) == -1
    assert call(ids=ctypes.c_void_p((1 << 20) + 4)) == -1    # int64 ids need 8 bytes
    assert call(W=ctypes.c_void_p((1 << 20) + 1)) == -1
    assert call(n=1 << 31) == -3
    assert call(V=(1 << 31) - 1) == -3
    assert call(d=(1 << 24) + 1) == -3


def test_embedding_backward_refusals():
    lib = nr.load()
    need = lib.nrnn_embedding_backward_workspace_bytes(100, 1000, 64)
    # two buffers of (id, position) pairs, V flags, partial sums of four chunks of 32
    assert need >= 4 * 100 * 4 + 1000 + 4 * 2 * 64 * 4
    assert lib.nrnn_embedding_backward_workspace_bytes(100, 0, 64) == 0
    assert lib.nrnn_embedding_backward_workspace_bytes(-1, 10, 64) == 0

    def call(ids=FAKE, g=FAKE, gW=FAKE, ws=WS, wsb=need, n=100, dtype=0):
        return lib.nrnn_embedding_backward(ids, 1, g, dtype, n, 1000, 64, -1, 1.0, 0, gW, ws, wsb, None)
    assert call(ws=None) == -7
    assert call(wsb=need - 1) == -7
    assert call(ws=ctypes.c_void_p((1 << 24) + 16)) == -7
    assert call(g=None) == -1
    assert call(gW=None) == -1
    assert call(ids=None) == -1
    assert call(dtype=-1) == -1
    assert call(g=ctypes.c_void_p((1 << 20) + 2)) == -1


def test_block_norm_refusals():
    f = nr.load().nrnn_block_norm_forward

    def call(x=FAKE, h=FAKE, gate=FAKE, dtype=0, rows=4, d=16, eps=1e-6, x_out=FAKE, u=FAKE):
        return f(x, h, gate, FAKE, FAKE, FAKE, dtype, rows, d, eps, x_out, u, None)
    assert call(rows=0) == 0
    assert call(dtype=5) == -1
    assert call(rows=-1) == -1
    assert call(d=0) == -1
    assert call(d=8193) == -3
    assert call(eps=-1.0) == -1
    assert call(eps=float("nan")) == -1
    assert call(x=None) == -1
    assert call(x_out=None) == -1
    assert call(h=None) == -1               # a gate without h
    assert call(h=None, gate=None, u=None) == -1
    assert call(h=ctypes.c_void_p((1 << 20) + 2)) == -1


def test_block_norm_backward_refusals():
    lib = nr.load()
    need = lib.nrnn_block_norm_backward_workspace_bytes(100, 64)
    assert need >= 3 * 64 * 4
    assert lib.nrnn_block_norm_backward_workspace_bytes(100, 8193) == 0

    def call(x=FAKE, h=FAKE, gate=FAKE, g_x=FAKE, g_u=FAKE, rows=100, d=64, gx=FAKE, gh=FAKE, gg=FAKE,
             ws=WS, wsb=BIG):
        return lib.nrnn_block_norm_backward(x, h, gate, None, None, None, g_x, g_u, 0, rows, d, 1e-6,
                                            gx, gh, gg, FAKE, FAKE, FAKE, ws, wsb, None)
    assert call(d=8193) == -3
    assert call(g_x=None, g_u=None) == -1
    assert call(h=None, gate=None, g_u=None) == -1
    assert call(h=None) == -1
    assert call(gx=None) == -1
    assert call(gh=None) == -1
    assert call(gg=None) == -1
    assert call(x=None) == -1
    assert call(ws=None) == -7
    assert call(wsb=need - 256) == -7


def test_vocab_loss_refusals():
    lib = nr.load()
    for back in (0, 1):
        need = lib.nrnn_vocab_loss_workspace_bytes(100, 64, 5000, 1, back)
        assert need > 100 * 64 * 2
        assert lib.nrnn_vocab_loss_workspace_bytes(100, 64, 5000, 0, back) > need   # three planes
        assert lib.nrnn_vocab_loss_workspace_bytes(100, 64, 0, 1, back) == 0
        assert lib.nrnn_vocab_loss_workspace_bytes(100, 64, 10, 9, back) == 0

        def call(x=FAKE, W=FAKE, t=FAKE, rows=100, d=64, V=5000, dtype=1, kind=1, a=FAKE, b=FAKE,
                 out=FAKE, ws=WS, wsb=BIG):
            if back:
                return lib.nrnn_vocab_loss_backward(x, W, dtype, rows, d, V, t, kind, -100, 1.0, a, b,
                                                    out, out, ws, wsb, None)
            return lib.nrnn_vocab_loss_forward(x, W, dtype, rows, d, V, t, kind, -100, 1.0, a, b, ws,
                                               wsb, None)
        assert call(dtype=3) == -1
        assert call(kind=3) == -1
        assert call(rows=-1) == -1
        assert call(d=0) == -1
        assert call(V=0) == -1
        assert call(x=None) == -1
        assert call(W=None) == -1
        assert call(t=None) == -1
        assert call(a=None) == -1
        assert call(W=ctypes.c_void_p((1 << 20) + 1)) == -1
        assert call(t=ctypes.c_void_p((1 << 20) + 4)) == -1
        assert call(V=(1 << 30) + 1) == -3
        assert call(ws=None) == -7
        assert call(wsb=1024) == -7
        assert call(ws=ctypes.c_void_p((1 << 24) + 128)) == -7
    assert lib.nrnn_vocab_loss_forward(None, FAKE, 1, 0, 64, 100, None, 1, -100, 1.0, None, None, None,
                                       0, None) == 0


def test_workspace_of_a_long_loss_stays_below_the_logits():
    """The backward keeps one piece of the vocabulary, not the rows x V array."""
    lib = nr.load()
    rows, V, d = 262144, 65536, 1024
    assert lib.nrnn_vocab_loss_workspace_bytes(rows, d, V, 1, 1) < rows * V * 2 / 4
    assert lib.nrnn_vocab_loss_workspace_bytes(rows, d, V, 1, 0) < rows * V * 2 / 4


def test_bindings_want_device_tensors():
    x, ids = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        nr.embedding(ids, x)
    with pytest.raises(ValueError):
        nr.embedding_backward(ids, x, 4)
    with pytest.raises(ValueError):
        nr.block_norm(x)
    with pytest.raises(ValueError):
        nr.block_norm_backward(x, g_u=x)
    with pytest.raises(ValueError):
        nr.vocab_loss(x, x, ids)
