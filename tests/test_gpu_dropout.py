"""Dropout against the generator restated in Python integers, and its statistics.

The mask is exact.  A kept value is one fp32 product (the scale itself rounded once)
and, with a residual, one fused addition: 2^-23 of the product plus the result's own
rounding."""
import math

import pytest
import torch

import nonlinear_rnn_gb300 as nr

pytestmark = pytest.mark.gpu

F64 = torch.float64
TYPES = [torch.float32, torch.bfloat16]


def philox(block, offset, seed):
    x = [block & 0xffffffff, block >> 32, offset & 0xffffffff, offset >> 32]
    k = [seed & 0xffffffff, seed >> 32]
    for _ in range(10):
        p, q = 0xD2511F53 * x[0], 0xCD9E8D57 * x[2]
        x = [q >> 32 ^ x[1] ^ k[0], q & 0xffffffff, p >> 32 ^ x[3] ^ k[1], p & 0xffffffff]
        k = [(k[0] + 0x9E3779B9) & 0xffffffff, (k[1] + 0xBB67AE85) & 0xffffffff]
    return x


def kept(n, p, seed, offset):
    words = [w for b in range((n + 3) // 4) for w in philox(b, offset, seed)][:n]
    return torch.tensor([w >= round(p * 2 ** 32) for w in words], device="cuda")


def test_the_generator_as_published():
    """Known answers of Philox 4x32 with ten rounds (all zeros; all ones)."""
    assert philox(0, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    ones = (1 << 64) - 1
    assert philox(ones, ones, ones) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("n", [1, 3, 4, 5, 8, 31, 1000, 4099])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(n, p, t):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x, res = torch.randn(n, generator=g, device="cuda").to(t), torch.randn(n, generator=g, device="cuda").to(t)
    seed, offset = 0x123456789abcdef0 + n, (1 << 40) + 7
    keep = kept(n, p, seed, offset)
    u = 2.0 ** -8 if t == torch.bfloat16 else 2.0 ** -24
    scaled = torch.where(keep, x.to(F64) / (1 - p) if p < 1 else 0.0, 0.0)
    for residual in (None, res):
        ref = scaled if residual is None else scaled + residual.to(F64)
        got = nr.dropout(x, p, seed, offset=offset, residual=residual)
        assert bool(((got.to(F64) - ref).abs() <= 2.0 ** -23 * scaled.abs() + u * ref.abs()).all())
        if residual is not None:
            assert torch.equal(got[~keep], residual[~keep])
        by_tensor = nr.dropout(x, p, torch.tensor([seed], device="cuda"), offset=offset, residual=residual)
        assert torch.equal(by_tensor, got)
    if p == 0.0:
        assert torch.equal(nr.dropout(x, p, seed), x)
    # in place, over x and over the residual; a view that is not 16-byte aligned
    a, b = x.clone(), res.clone()
    want = nr.dropout(x, p, seed, residual=res)
    assert nr.dropout(a, p, seed, residual=res, out=a) is a and torch.equal(a, want)
    nr.dropout(x, p, seed, residual=b, out=b)
    assert torch.equal(b, want)
    shifted = torch.cat([x[:1], x])[1:]
    assert torch.equal(nr.dropout(shifted, p, seed, residual=res), want)


def test_what_is_dropped_is_zero():
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    keep = kept(4096, 0.5, 5, 0)
    y = nr.dropout(x, 0.5, 5)
    assert torch.equal(y[~keep], torch.zeros_like(y[~keep])) and not bool(y[keep].isfinite().any())
    assert torch.equal(nr.dropout(x, 1.0, 5), torch.zeros_like(x))


def test_the_gradient_is_the_same_call():
    """sum(g dropout(x)) is linear in x: its slope along any direction is that of the call on g."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, up, way = (torch.randn(50, 33, generator=g, device="cuda") for _ in range(3))
    gx = nr.dropout(up, 0.3, 77, offset=2)
    f = [(nr.dropout(x + s * way, 0.3, 77, offset=2).to(F64) * up).sum() for s in (0.5, -0.5)]
    slope, ours = float(f[0] - f[1]), float((gx.to(F64) * way).sum())
    assert abs(slope - ours) <= 1650 * 2.0 ** -22 * 12    # roundings of 1650 products of a few units each


@pytest.mark.parametrize("p", [0.1, 0.5])
def test_rates_and_independence(p):
    """Shares of kept elements within five standard deviations, over elements, offsets and seeds."""
    n = 1 << 20
    x = torch.ones(n, device="cuda")
    masks = [nr.dropout(x, p, s, offset=o) > 0 for s, o in ((1, 0), (2, 0), (1, 1), (1, 1 << 32), (1 + (1 << 32), 0))]
    sd = math.sqrt(p * (1 - p) / n)
    for m in masks:
        assert abs(float(m.double().mean()) - (1 - p)) < 5 * sd
    for i, a in enumerate(masks):
        for b in masks[i + 1:]:
            q = p * (1 - p) * 2                           # probability that two masks differ
            assert abs(float((a != b).double().mean()) - q) < 5 * math.sqrt(q * (1 - q) / n)
    neighbours = float((masks[0][1:] != masks[0][:-1]).double().mean())
    assert abs(neighbours - 2 * p * (1 - p)) < 6 * math.sqrt(0.25 / n) * 2


def test_elements_beyond_32_bits():
    n = (1 << 32) + 64
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = nr.dropout(x, 0.5, 3, out=x)
    tail = (y[-64:] > 0).cpu().tolist()
    words = [w for b in range((1 << 30), (1 << 30) + 16) for w in philox(b, 0, 3)]
    assert tail == [w >= 1 << 31 for w in words]
    del x, y


def test_captured_with_a_seed_on_the_device():
    x = torch.ones(1000, device="cuda")
    seed = torch.tensor([5], device="cuda")
    nr.dropout(x, 0.5, seed)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = nr.dropout(x, 0.5, seed)
    for s in (5, 6, -7):
        seed.fill_(s)
        graph.replay()
        assert torch.equal(y, nr.dropout(x, 0.5, s))


def test_refusals():
    x = torch.ones(8, device="cuda")
    for call in (lambda: nr.dropout(x.cpu(), 0.1, 1), lambda: nr.dropout(x, -0.1, 1), lambda: nr.dropout(x, 1.5, 1),
                 lambda: nr.dropout(x, float("nan"), 1), lambda: nr.dropout(x, 0.1, 1, residual=x[:4]),
                 lambda: nr.dropout(x, 0.1, torch.ones(2, dtype=torch.int64, device="cuda")),
                 lambda: nr.dropout(x, 0.1, torch.ones(1, dtype=torch.int64)),
                 lambda: nr.dropout(x, 0.1, 1, out=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nr.dropout(x.double(), 0.1, 1)
    y = torch.ones(16, device="cuda")
    with pytest.raises(ValueError):
        nr.dropout(y[:8], 0.1, 1, out=y[4:12])            # reaches into x from another place
    assert nr.dropout(x[:0], 0.1, 1).numel() == 0
