"""Host-side checks of the block's operators: workspace sizes and the refusals,
which come before any launch.  No GPU needed."""
import ctypes

import pytest
import torch

import nonlinear_rnn_gb300 as nr


def at(n):
    return ctypes.c_void_p(n)   # never dereferenced: the checks fail first


FAKE, WS, BIG = at(1 << 20), at(1 << 40), 1 << 50


def test_linear_recurrence_refusals():
    lib = nr.load()
    size = lib.nrnn_linear_recurrence_workspace_bytes
    assert size(2, 100, 64, 1, 0, 1) >= size(2, 100, 64, 1, 0, 0) > 0
    assert size(2, 100, 0, 1, 0, 0) == 0
    assert size(-1, 100, 64, 1, 0, 0) == 0
    assert size(2, 100, 64, 3, 0, 0) == 0
    # buffers of a pack of three segments of 8 steps of 16 units, well apart
    P, H, gH, gP, state, last = (at(i << 24) for i in range(1, 7))

    def forward(P=P, dtype=0, prm=FAKE, B=1, T=8, d=16, cu=None, S=0, state=state, H=H, last=last, ws=WS, wsb=BIG):
        return lib.nrnn_linear_recurrence_forward(P, dtype, prm, B, T, d, cu, S, state, H, last, ws, wsb, None)

    def backward(P=P, dtype=0, prm=FAKE, B=1, T=8, d=16, cu=None, S=0, state=state, H=H, gH=gH, g_last=state, gP=gP,
                 gprm=at(8 << 24), g_state=last, ws=WS, wsb=BIG):
        return lib.nrnn_linear_recurrence_backward(P, dtype, prm, B, T, d, cu, S, state, H, gH, g_last, gP, gprm, g_state,
                                                   ws, wsb, None)
    for call in (forward, backward):
        assert call(dtype=2) == -1
        assert call(B=-1) == -1
        assert call(T=-1) == -1
        assert call(d=0) == -1
        assert call(d=12) == -3
        assert call(d=(1 << 24) + 8) == -3
        assert call(T=1 << 31) == -3
        assert call(B=2, cu=FAKE, S=2) == -2
        assert call(cu=FAKE, S=0) == -2
        assert call(P=None) == -1
        assert call(prm=None) == -1
        assert call(H=None) == -1
        assert call(P=at((1 << 24) + 8)) == -1
        assert call(H=at((2 << 24) + 8)) == -1
        assert call(state=at((5 << 24) + 4)) == -1
        assert call(ws=None) == -7
        assert call(ws=at((1 << 40) + 64)) == -7
        assert call(wsb=16) == -7
    assert forward(H=at((1 << 24) + 64)) == -1                   # inside preact
    assert forward(last=at((5 << 24) + 16)) == -1                # part of state
    assert backward(gH=None) == -1
    assert backward(gP=None) == -1
    assert backward(gprm=None) == -1
    assert backward(gP=H) == -1
    assert backward(gP=P) == -1

    def step(P=P, dtype=0, prm=FAKE, slots=4, d=16, state=state, h=H, out=last):
        return lib.nrnn_linear_recurrence_step(P, dtype, prm, slots, d, state, h, out, None)
    assert step(slots=0) == 0
    assert step(slots=-1) == -1
    assert step(dtype=9) == -1
    assert step(d=20) == -3
    assert step(P=None) == -1
    assert step(h=None) == -1
    assert step(out=None) == -1
    assert step(h=P) == -1
    assert step(out=at((5 << 24) + 64)) == -1                    # part of state
    assert step(h=state) == -1


@pytest.mark.parametrize("dtype", [0, 1])
def test_gated_mlp_refusals(dtype):
    lib = nr.load()
    kept, size = lib.nrnn_gated_mlp_kept_bytes, lib.nrnn_gated_mlp_workspace_bytes
    assert kept(100, 24, dtype) >= 3 * 100 * 24 * (2 if dtype else 4)
    assert size(100, 16, 24, dtype, 0) > 0 and size(100, 16, 24, dtype, 1) > 0
    assert kept(100, 0, dtype) == kept(-1, 24, dtype) == kept(1, 24, 5) == 0
    assert size(100, 0, 24, dtype, 0) == size(100, 16, 24, 7, 1) == size((1 << 30) + 1, 16, 24, dtype, 0) == 0
    assert size(100, 16, 24, dtype, 3) == size(100, 16, 24, dtype, -1) == 0 < size(4, 16, 24, dtype, 0) < size(4, 16, 24, dtype, 2)

    def forward(x=FAKE, Wi=FAKE, Wo=FAKE, dtype=dtype, n=100, d=16, f=24, y=at(1 << 24), kept=WS, ws=WS, wsb=BIG):
        return lib.nrnn_gated_mlp_forward(x, Wi, Wo, dtype, n, d, f, y, kept, ws, wsb, None)

    def backward(x=FAKE, Wi=FAKE, Wo=FAKE, dtype=dtype, n=100, d=16, f=24, kept=WS, g=FAKE, gx=at(1 << 24),
                 gWi=at(2 << 24), gWo=at(3 << 24),
                 ws=WS, wsb=BIG):
        return lib.nrnn_gated_mlp_backward(x, Wi, Wo, kept, g, dtype, n, d, f, gx, gWi, gWo, ws, wsb, None)
    for call in (forward, backward):
        assert call(dtype=2) == -1
        assert call(n=-1) == -1
        assert call(d=0) == -1
        assert call(f=0) == -1
        assert call(n=(1 << 30) + 1) == -3
        assert call(d=(1 << 20) + 1) == -3
        assert call(f=(1 << 20) + 1) == -3
        assert call(x=None) == -1
        assert call(Wi=None) == -1
        assert call(Wo=at((1 << 20) + 1)) == -1
        assert call(kept=at((1 << 40) + 16)) == -1
        assert call(ws=None) == -7
        assert call(ws=at((1 << 40) + 16)) == -7
        assert call(wsb=16) == -7
    assert forward(n=0) == 0
    assert forward(y=None) == -1
    assert backward(kept=None) == -1
    assert backward(g=None) == -1
    assert backward(gx=None) == -1
    assert backward(gWi=None) == -1
    assert backward(gWo=at((1 << 20) + 1)) == -1


def test_dropout_refusals():
    f = nr.load().nrnn_dropout

    def call(x=FAKE, dtype=1, n=64, p=0.1, seed_at=None, residual=None, out=at(1 << 24)):
        return f(x, dtype, n, p, 1, seed_at, 0, residual, out, None)
    assert call(n=0) == 0
    assert call(dtype=2) == -1
    assert call(n=-1) == -1
    assert call(n=(1 << 48) + 1) == -3
    assert call(p=-0.1) == -1
    assert call(p=1.01) == -1
    assert call(p=float("nan")) == -1
    assert call(x=None) == -1
    assert call(out=None) == -1
    assert call(x=at((1 << 20) + 1)) == -1
    assert call(residual=at((1 << 20) + 1)) == -1
    assert call(seed_at=at((1 << 20) + 4)) == -1
    assert call(out=at((1 << 20) + 64)) == -1                    # reaches into x
    assert call(residual=at((1 << 24) - 64)) == -1


def test_bindings_want_device_tensors():
    P, x = torch.zeros(1, 4, 24), torch.zeros(4, 8)
    for call in (lambda: nr.linear_recurrence(P, torch.zeros(3, 8)), lambda: nr.linear_recurrence_step(torch.zeros(3, 8), None, P[0]),
                 lambda: nr.linear_recurrence_backward(P, torch.zeros(3, 8), P, P), lambda: nr.dropout(x, 0.1, 1),
                 lambda: nr.gated_mlp(x, torch.zeros(6, 8), torch.zeros(8, 3)),
                 lambda: nr.gated_mlp_backward(x, torch.zeros(6, 8), torch.zeros(8, 3), x, x)):
        with pytest.raises(ValueError):
            call()


def test_recurrence_outputs_apart():
    """Every output against every input and every other output, at equal and at
    partly covered addresses: 3 x 8 steps of 16 units in fp32."""
    lib = nr.load()
    names = ("P", "prm", "state", "H", "gH", "g_last", "gP", "gprm", "g_state", "last")
    far = {k: (i + 1) << 24 for i, k in enumerate(names)}

    def forward(**k):
        a = {n: at(v) for n, v in {**far, **k}.items()}
        return lib.nrnn_linear_recurrence_forward(a["P"], 0, a["prm"], 3, 8, 16, None, 0, a["state"], a["H"], a["last"], WS,
                                                  16, None)

    def backward(**k):
        a = {n: at(v) for n, v in {**far, **k}.items()}
        return lib.nrnn_linear_recurrence_backward(a["P"], 0, a["prm"], 3, 8, 16, None, 0, a["state"], a["H"], a["gH"],
                                                   a["g_last"], a["gP"], a["gprm"], a["g_state"], WS, 16, None)
    assert forward() == backward() == -7                         # only the workspace is too small
    for call, outs, ins in ((forward, ("H", "last"), ("P", "prm", "state")),
                            (backward, ("gP", "gprm", "g_state"), ("P", "prm", "state", "H", "gH", "g_last"))):
        for o in outs:
            for other in (*ins, *(p for p in outs if p != o)):
                assert call(**{o: far[other]}) == -1, (o, other)
                assert call(**{o: far[other] + 64}) == -1, (o, other)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("n", [4, 100])
def test_gated_mlp_outputs_apart(dtype, n):
    """The same of the feed-forward block, at a decode step's rows and more."""
    lib = nr.load()
    names = ("x", "Wi", "Wo", "kept", "g", "y", "gx", "gWi", "gWo")
    far = {k: (i + 1) << 24 for i, k in enumerate(names)}

    def forward(**k):
        a = {m: at(v) for m, v in {**far, **k}.items()}
        return lib.nrnn_gated_mlp_forward(a["x"], a["Wi"], a["Wo"], dtype, n, 64, 128, a["y"], a["kept"], WS, 16, None)

    def backward(**k):
        a = {m: at(v) for m, v in {**far, **k}.items()}
        return lib.nrnn_gated_mlp_backward(a["x"], a["Wi"], a["Wo"], a["kept"], a["g"], dtype, n, 64, 128, a["gx"], a["gWi"],
                                           a["gWo"], WS, 16, None)
    assert forward() == backward() == -7
    for call, outs, ins in ((forward, ("y", "kept"), ("x", "Wi", "Wo")),
                            (backward, ("gx", "gWi", "gWo"), ("x", "Wi", "Wo", "kept", "g"))):
        for o in outs:
            for other in (*ins, *(p for p in outs if p != o)):
                assert call(**{o: far[other]}) == -1, (o, other)
                assert call(**{o: far[other] + 256}) == -1, (o, other)
