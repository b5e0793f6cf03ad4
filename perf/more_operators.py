"""What a block of a recurrent language model needs besides the operators of
``operators.py``, as cases to run.

Three operators: the gated linear recurrence (forward, gradient and the step of
one token per slot), the gated feed-forward block with its gradient, and dropout
whose mask is made again from a counter instead of being stored.  ``run``
computes a case with the library's kernels (``own``) or in plain fp32 torch
operations, and ``exact`` gives the same outputs from the definitions in float64.

Shapes follow the recurrent layer's own workloads (4 x 131072 x 64, 8 x 4096 x
256, 16 x 16384 x 1024, the ragged pack of 262144 x 512); the feed-forward block
is four times as wide as the model, or of sizes that no tile divides."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
#: elements of the largest listed activations
MOST_UNITS = 16 * 16384 * 1024
#: rows x width x inner width of the largest listed feed-forward step
MOST_MLP = 32768 * 1024 * 4096


def listed():
    return [
        # one decode step of the recurrence, 16 slots
        {"name": "rec_step", "op": "rec", "way": "step", "type": "bf16", "b": 16, "t": 1, "d": 1024, "segments": 0, "state": True},
        # a decode step of a full batch of slots, fp32
        {"name": "rec_step_wide_f32", "op": "rec", "way": "step", "type": "f32", "b": 8192, "t": 1, "d": 512, "segments": 0, "state": True},
        # the forward over long sequences of a narrow layer
        {"name": "rec_long_f32", "op": "rec", "way": "forward", "type": "f32", "b": 4, "t": 131072, "d": 64, "segments": 0, "state": False},
        # the forward of a training batch
        {"name": "rec_bf16", "op": "rec", "way": "forward", "type": "bf16", "b": 16, "t": 16384, "d": 1024, "segments": 0, "state": False},
        # the gradient of a ragged pack that continues earlier text
        {"name": "rec_grad_pack_f32", "op": "rec", "way": "backward", "type": "f32", "b": 1, "t": 262144, "d": 512, "segments": 64, "state": True},
        # the gradient of a batch whose length and width no tile divides
        {"name": "rec_grad_odd_bf16", "op": "rec", "way": "backward", "type": "bf16", "b": 7, "t": 3001, "d": 264, "segments": 0, "state": True},
        # the gradient of a training batch
        {"name": "rec_grad_bf16", "op": "rec", "way": "backward", "type": "bf16", "b": 16, "t": 16384, "d": 1024, "segments": 0, "state": False},
        # the feed-forward block of one decode step of 8 slots
        {"name": "mlp_step", "op": "mlp", "way": "forward", "type": "bf16", "n": 8, "d": 1024, "f": 4096},
        # a training step of an odd fp32 batch
        {"name": "mlp_odd_f32", "op": "mlp", "way": "train", "type": "f32", "n": 1501, "d": 250, "f": 683},
        # a training step of 32768 tokens
        {"name": "mlp_bf16", "op": "mlp", "way": "train", "type": "bf16", "n": 32768, "d": 1024, "f": 4096},
        # dropout of an odd fp32 batch, no residual
        {"name": "drop_odd_f32", "op": "drop", "type": "f32", "n": 4099, "d": 250, "p": 0.1, "residual": False},
        # dropout of a block's output and its addition to the residual stream
        {"name": "drop_bf16", "op": "drop", "type": "bf16", "n": 262144, "d": 1024, "p": 0.1, "residual": True},
    ]


def spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def width(rng, low, high):
    """A width: one in two divides by 64, as layers' widths do; the others fall anywhere."""
    d = spread(rng, low, high)
    return d if rng.random() < 0.5 else max(low, d // 64 * 64)


def draw(rng):
    kind = rng.choice(("rec", "rec", "mlp", "mlp", "drop"))
    case = {"op": kind, "type": rng.choice(("bf16", "f32"))}
    if kind == "mlp":
        # six products of planes make an fp32 product
        most = MOST_MLP // (1 if case["type"] == "bf16" else 6)
        d, f = width(rng, 64, 1024), width(rng, 128, 4096)
        return {**case, "way": rng.choice(("forward", "train")), "n": spread(rng, 1, min(32768, most // (d * f))), "d": d, "f": f}
    most = MOST_UNITS // (1 if case["type"] == "bf16" else 2)
    if kind == "drop":
        d = width(rng, 64, 1024)
        return {**case, "n": spread(rng, 1, most // d), "d": d, "p": rng.choice((0.05, 0.1, 0.5)), "residual": rng.random() < 0.5}
    d = width(rng, 32, 1024) // 8 * 8            # units come in groups of 8
    case.update(way=rng.choice(("forward", "backward", "step")), d=d, segments=0, state=True)
    if case["way"] == "step":
        return {**case, "b": spread(rng, 1, 8192), "t": 1}
    case["state"] = rng.random() < 0.5
    if rng.random() < 0.4:                       # a pack
        t = spread(rng, 64, min(262144, most // d))
        return {**case, "b": 1, "t": t, "segments": spread(rng, 1, min(256, t // 16))}
    b = spread(rng, 1, 16)
    return {**case, "b": b, "t": spread(rng, 1, min(131072, most // (b * d)))}


def bounds(g, t, segments):
    """Offsets of a pack of uneven segments, some of them empty."""
    share = torch.rand(segments, generator=g).double() + 0.05
    if segments > 3:
        share[torch.rand(segments, generator=g) < 0.05] = 0.0
        share[segments // 2] = 1.0
    ends = (share.cumsum(0) / share.sum() * t).round().long().clamp_(0, t)
    ends[-1] = t
    return torch.cat([torch.zeros(1, dtype=torch.long), ends]).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    d, t = case["d"], TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"op": case["op"], "way": case.get("way")}
    if case["op"] == "mlp":
        n, f = case["n"], case["f"]
        s["x"] = normal(n, d)                                   # normalised rows
        s["W_in"] = normal(2 * f, d, std=1 / math.sqrt(d))
        s["W_out"] = normal(d, f, std=1 / math.sqrt(f))
        if case["way"] == "train":
            s["g"] = normal(n, d, std=0.1)
        return s
    if case["op"] == "drop":
        s["x"] = normal(case["n"], d)
        s["residual"] = normal(case["n"], d, std=2.0) if case["residual"] else None
        s.update(p=case["p"], seed=int(seed) * 0x9E3779B97F4A7C15 % 2 ** 63, offset=int(seed) % 1000)
        return s
    b, steps = case["b"], case["t"]
    # the slowest decay of a unit, at an open gate, is 0.9 to 0.999 in the eighth root
    slow = torch.rand(d, generator=g, device="cuda") * 0.099 + 0.9
    s["params"] = torch.stack([-8 * slow.log(), normal(d, std=0.5, dtype=torch.float32), normal(d, std=0.5, dtype=torch.float32)])
    s["cu"], rows = None, b
    if case["segments"]:
        host = torch.Generator()
        host.manual_seed(int(seed))
        cu = bounds(host, steps, case["segments"])
        s["cu"], rows = cu.cuda(), case["segments"]
        if own:
            import nonlinear_rnn_gb300 as nr

            s["pack"] = nr.DeviceCuSeqlens(cu, steps)
    s["state"] = normal(rows, d, std=0.5, dtype=torch.float32) if case["state"] else None
    if case["way"] == "step":
        s["P"] = normal(b, 3 * d)
        return s
    s["P"] = normal(b, steps, 3 * d)
    if case["way"] == "backward":
        s["H"] = plain_scan(s)[0].to(t)                         # as the forward left it
        s["gH"] = normal(b, steps, d, std=0.1)
        s["g_state"] = normal(rows, d, std=0.1, dtype=torch.float32) if case["state"] else None
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import nonlinear_rnn_gb300 as nr

    if s["op"] == "drop":
        return {"y": nr.dropout(s["x"], s["p"], s["seed"], offset=s["offset"], residual=s["residual"])}
    if s["op"] == "mlp":
        if s["way"] == "forward":
            return {"y": nr.gated_mlp(s["x"], s["W_in"], s["W_out"])}
        y, kept = nr.gated_mlp(s["x"], s["W_in"], s["W_out"], keep=True)
        gx, gW_in, gW_out = nr.gated_mlp_backward(s["x"], s["W_in"], s["W_out"], kept, s["g"])
        return {"y": y, "gx": gx, "gW_in": gW_in, "gW_out": gW_out}
    if s["way"] == "step":
        h, state = nr.linear_recurrence_step(s["params"], s["state"], s["P"])
        return {"h": h, "state": state}
    pack = s["pack"] if s["cu"] is not None else None
    if s["way"] == "forward":
        H, state = nr.linear_recurrence(s["P"], s["params"], cu_seqlens=pack, state=s["state"])
        return {"H": H, "state": state}
    r = nr.linear_recurrence_backward(s["P"], s["params"], s["H"], s["gH"], cu_seqlens=pack, state=s["state"], g_state=s["g_state"])
    return {"gP": r.gP, "gparams": r.gparams, "g_state": r.g_state}


def run_plain(s):
    t = s["x" if "x" in s else "P"].dtype
    if s["op"] == "drop":
        e = s["x"].numel()
        kept = plain_words(e, s["seed"], s["offset"]) >= round(s["p"] * 2 ** 32)
        y = torch.where(kept.view(s["x"].shape), s["x"].float() * (1 / (1 - s["p"])), 0.0)
        return {"y": (y if s["residual"] is None else s["residual"].float() + y).to(t)}
    if s["op"] == "mlp":
        x, W_in, W_out = s["x"].float(), s["W_in"].float(), s["W_out"].float()
        f = W_out.shape[1]
        ab = x @ W_in.T
        a, b = ab[:, :f], ab[:, f:]
        sig = 1 / (1 + (-a).exp())
        m = a * sig * b
        out = {"y": (m @ W_out.T).to(t)}
        if s["way"] == "train":
            g = s["g"].float()
            out["gW_out"] = (g.T @ m).to(t)
            del m
            gm = g @ W_out
            gab = torch.cat([gm * b * (sig * (1 + a * (1 - sig))), gm * (a * sig)], 1)
            out["gx"], out["gW_in"] = (gab @ W_in).to(t), (gab.T @ x).to(t)
        return out
    if s["way"] == "step":
        _, a, i, q = plain_gates(s["P"].float(), s["params"])
        v = s["P"].float()[:, 2 * s["params"].shape[1]:]
        h = a * s["state"] + q * i * v
        return {"h": h.to(t), "state": h}
    if s["way"] == "forward":
        H, state = plain_scan(s)
        return {"H": H.to(t), "state": state}
    return plain_backward(s)


def plain_gates(P, params):
    """r, the decay a, the input gate i, and sqrt(1 - a^2)."""
    d = params.shape[1]
    rate, b_a, b_i = params
    r = 1 / (1 + (-(P[..., :d] + b_a)).exp())
    i = 1 / (1 + (-(P[..., d:2 * d] + b_i)).exp())
    w = -rate * r
    return r, w.exp(), i, (-(2 * w).expm1()).sqrt()


def doubling(a, u):
    """h_t = a_t h_{t-1} + u_t along axis 1, h = 0 before: spans of twice the length in turn."""
    step = 1
    while step < u.shape[1]:
        u[:, step:] += a[:, step:] * u[:, :-step].clone()
        a[:, step:] *= a[:, :-step].clone()
        step *= 2
    return u


def plain_ends(s):
    """First and last rows of the sequences in a (B T)-row array, and which sequences are not empty."""
    b, t = s["P"].shape[:2]
    if s["cu"] is not None:
        cu = s["cu"].long()
        return cu[:-1], cu[1:] - 1, cu[1:] > cu[:-1]
    first = torch.arange(b, device="cuda") * t
    return first, first + t - 1, torch.full((b,), t > 0, device="cuda")


def plain_scan(s):
    """H in fp32 and the last states."""
    b, t = s["P"].shape[:2]
    d = s["params"].shape[1]
    P = s["P"].float()
    _, a, i, q = plain_gates(P, s["params"])
    u = q.mul_(i).mul_(P[..., 2 * d:])
    del P, i
    first, last, some = plain_ends(s)
    af, uf = a.view(-1, d), u.view(-1, d)
    if s["state"] is not None:
        uf[first[some]] += af[first[some]] * s["state"][some]
    af[first[some]] = 0.0
    H = doubling(a, u)
    state = torch.zeros(len(first), d, device="cuda") if s["state"] is None else s["state"].clone()
    state[some] = H.view(-1, d)[last[some]]
    return H, state


def plain_backward(s):
    t = s["P"].dtype
    d = s["params"].shape[1]
    P, H = s["P"].float(), s["H"].float()
    r, a, i, q = plain_gates(P, s["params"])
    first, last, some = plain_ends(s)
    before = torch.cat([torch.zeros_like(H[:, :1]), H[:, :-1]], 1)
    before.view(-1, d)[first[some]] = 0.0 if s["state"] is None else s["state"][some]
    G = s["gH"].float().clone()
    if s["g_state"] is not None:
        G.view(-1, d)[last[some]] += s["g_state"][some]
    # G_t += a_{t+1} G_{t+1} inside a sequence
    after = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    after.view(-1, d)[last[some]] = 0.0
    G = doubling(after.flip(1), G.flip(1)).flip(1)
    del after
    v = P[..., 2 * d:]
    w = G * (a * before - torch.where(q > 0, a * a / q, 0.0) * i * v)
    rate = s["params"][0]
    g_a, g_i = -w * rate * r * (1 - r), G * q * v * i * (1 - i)
    gP = torch.cat([g_a, g_i, G * q * i], 2).to(t)
    sums = torch.stack([-(w * r).sum((0, 1)), g_a.sum((0, 1)), g_i.sum((0, 1))])
    out = {"gP": gP, "gparams": sums, "g_state": None}
    if s["state"] is not None:
        g_state = s["g_state"].clone()                          # an empty sequence hands its state on
        g_state[some] = (a * G).view(-1, d)[first[some]]
        out["g_state"] = g_state
    return out


MASK = 0xFFFFFFFF


def high_word(m, x):
    """The upper 32 bits of a product of two 32-bit numbers, held in int64."""
    return (m * (x >> 16) + (m * (x & 0xFFFF) >> 16)) >> 16


def plain_words(n, seed, offset):
    """n 32-bit words: counter (block, offset), key seed, ten Philox rounds for four words."""
    block = torch.arange((n + 3) // 4, device="cuda")
    x0, x1 = block & MASK, block >> 32
    x2, x3 = torch.full_like(block, offset & MASK), torch.full_like(block, offset >> 32)
    k0, k1 = seed & MASK, seed >> 32
    for _ in range(10):
        h0, h1 = high_word(0xD2511F53, x0), high_word(0xCD9E8D57, x2)
        l0, l1 = x0 * 0xD2511F53 & MASK, x2 * 0xCD9E8D57 & MASK
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK, (k1 + 0xBB67AE85) & MASK
    return torch.stack([x0, x1, x2, x3], 1).view(-1)[:n]


def work(case):
    es, d = (2 if case["type"] == "bf16" else 4), case["d"]
    if case["op"] == "drop":
        n = case["n"] * d
        return {"bytes": es * n * (3 if case["residual"] else 2), "flops": n * 3}
    if case["op"] == "mlp":
        n, f = case["n"], case["f"]
        if case["way"] == "forward":
            return {"bytes": es * d * (2 * n + 3 * f), "flops": 6 * n * d * f}
        # x, g and the weights in; y, gx and the weights' gradients out
        return {"bytes": es * d * (4 * n + 6 * f), "flops": 18 * n * d * f}
    n = case["b"] * case["t"] * d
    rows = (case["segments"] or case["b"]) * d
    if case["way"] == "step":
        return {"bytes": n * (4 * es + 8) + 12 * d, "flops": 20 * n}
    states = rows * 4 * (1 + bool(case["state"]))
    if case["way"] == "forward":
        return {"bytes": 4 * es * n + states + 12 * d, "flops": 20 * n}
    # P, H and gH in, gP out
    return {"bytes": 8 * es * n + 24 * d + rows * 12 * bool(case["state"]), "flops": 45 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "drop":
        return {"y": exact_dropout(s)}
    return exact_mlp(case, s) if case["op"] == "mlp" else exact_recurrence(case, s)


def exact_mlp(case, s):
    if (18 if case["way"] == "train" else 6) * case["n"] * case["d"] * case["f"] > 1.1e13:   # about 20 s of fp64
        return None
    f64, f = torch.float64, case["f"]
    W_in, W_out = s["W_in"].to(f64), s["W_out"].to(f64)
    train = case["way"] == "train"
    parts, gW_in, gW_out = [], torch.zeros_like(W_in), torch.zeros_like(W_out)
    for r in range(0, case["n"], 4096):
        x = s["x"][r:r + 4096].to(f64)
        pre = torch.matmul(x, W_in.t()).requires_grad_(train)
        m = torch.nn.functional.silu(pre[:, :f]) * pre[:, f:]
        y = torch.matmul(m.detach(), W_out.t())
        if not train:
            parts.append((y,))
            continue
        g = s["g"][r:r + 4096].to(f64)
        g_pre, = torch.autograd.grad(m, pre, torch.matmul(g, W_out))
        gW_out.addmm_(g.t(), m.detach())
        gW_in.addmm_(g_pre.t(), x)
        parts.append((y, torch.matmul(g_pre, W_in)))
    cat = [torch.cat(c) for c in zip(*parts)]
    return {"y": cat[0]} if not train else {"y": cat[0], "gx": cat[1], "gW_in": gW_in, "gW_out": gW_out}


def exact_dropout(s):
    """Rows in turn; the generator on 16-bit digits held in float64."""
    x = s["x"]
    flat, base = x.reshape(-1), None if s["residual"] is None else s["residual"].reshape(-1)
    y = torch.empty(flat.numel(), dtype=torch.float64, device="cuda")
    limit = round(s["p"] * 2 ** 32)

    def product(m, w):
        """(high, low) words of m w."""
        low = m % 65536 * w                       # below 2^48
        high = m // 65536 * w
        total = high + torch.floor(low / 65536)   # below 2^49: both exact
        top = torch.floor(total / 65536)
        return top, (total - top * 65536) * 65536 + torch.remainder(low, 65536)

    def mix(*words):
        out = words[0].long()
        for w in words[1:]:
            out = out.bitwise_xor(w.long() if torch.is_tensor(w) else torch.full_like(out, w))
        return out.double()

    for at in range(0, flat.numel(), 1 << 25):
        n = min(1 << 25, flat.numel() - at)
        c = (torch.arange((n + 3) // 4, device="cuda") + at // 4).double()
        c = [torch.remainder(c, 2.0 ** 32), torch.floor(c / 2.0 ** 32), torch.full_like(c, s["offset"] % 2 ** 32), torch.full_like(c, s["offset"] // 2 ** 32)]
        key = [s["seed"] % 2 ** 32, s["seed"] // 2 ** 32]
        for turn in range(10):
            (h0, l0), (h1, l1) = product(0xD2511F53, c[0]), product(0xCD9E8D57, c[2])
            c = [mix(h1, c[1], key[0]), l1, mix(h0, c[3], key[1]), l0]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        word = torch.stack(c, 1).reshape(-1)[:n]
        y[at:at + n] = torch.where(word >= limit, flat[at:at + n].double() / (1 - s["p"]), torch.zeros((), dtype=torch.float64, device="cuda"))
        if base is not None:
            y[at:at + n] += base[at:at + n].double()
    return y.view(x.shape)


def exact_recurrence(case, s):
    """One step of time after another in float64, packs as a padded batch of their segments; the
    gates' gradients by torch's differentiation."""
    f64, d = torch.float64, case["d"]
    if case["way"] == "step":
        a, u = exact_step(s["P"].to(f64), *s["params"].to(f64))
        h = torch.addcmul(u, a, s["state"].to(f64))
        return {"h": h, "state": h.clone()}
    b, t = s["P"].shape[:2]
    if s["cu"] is None:
        lengths = [t] * b
        starts = [i * t for i in range(b)]
    else:
        cu = s["cu"].tolist()
        lengths = [e - f for f, e in zip(cu, cu[1:])]
        starts = cu[:-1]
    longest, rows = max(lengths), len(lengths)
    if longest * rows * d > 4 * MOST_UNITS:
        return None
    at = torch.arange(longest, device="cuda")
    length = torch.tensor(lengths, device="cuda")
    inside = at[None] < length[:, None]
    index = torch.where(inside, at[None] + torch.tensor(starts, device="cuda")[:, None], 0)
    P = s["P"].view(b * t, 3 * d)
    weights = s["params"].to(f64)
    state = torch.zeros(rows, d, dtype=f64, device="cuda") if s["state"] is None else s["state"].to(f64)
    span = max(1, (1 << 24) // (rows * d))        # steps of time whose gates are at hand at once
    if case["way"] == "forward":
        H, h = torch.zeros(b * t, d, dtype=f64, device="cuda"), state
        for t0 in range(0, longest, span):
            where = index[:, t0:t0 + span]
            a, u = exact_step(P[where].to(f64), *weights)
            ok = inside[:, t0:t0 + span]
            got = []
            for j in range(where.shape[1]):
                h = torch.where(ok[:, j, None], torch.addcmul(u[:, j], a[:, j], h), h)
                got.append(h)
            H[where[ok]] = torch.stack(got, 1)[ok]
        return {"H": H.view(b, t, d), "state": h}
    gH, H = s["gH"].view(b * t, d), s["H"].view(b * t, d)
    carry = torch.zeros_like(state) if s["g_state"] is None else s["g_state"].to(f64)   # dL/dh from what comes later
    gP, sums = torch.empty(b * t, 3 * d, dtype=f64, device="cuda"), torch.zeros(3, d, dtype=f64, device="cuda")
    for t0 in reversed(range(0, longest, span)):
        where, ok = index[:, t0:t0 + span], inside[:, t0:t0 + span]
        p = P[where].to(f64).requires_grad_(True)
        w = [x.clone().requires_grad_(True) for x in weights]
        a, u = exact_step(p, *w)
        back = H[(where - 1).clamp_(min=0)].to(f64)
        if t0 == 0:
            back[:, 0] = state
        with torch.no_grad():
            up = torch.where(ok[..., None], gH[where].to(f64), 0.0)
            got = []
            for j in reversed(range(where.shape[1])):
                total = torch.where(ok[:, j, None], up[:, j] + carry, 0.0)
                got.append(total)
                carry = torch.where(ok[:, j, None], a[:, j] * total, carry)
            G = torch.stack(got[::-1], 1)
        gp, *gw = torch.autograd.grad([a, u], [p, *w], [G * back, G])
        gP[where[ok]] = gp[ok]
        sums += torch.stack(gw)
    return {"gP": gP.view(b, t, 3 * d), "gparams": sums, "g_state": None if s["state"] is None else carry}


def exact_step(P, rate, b_a, b_i):
    """(a, u) of h = a h + u from preactivations."""
    f, i, v = P.chunk(3, -1)
    fall = rate * torch.sigmoid(f + b_a)
    # 1 - a^2 = (1 - a)(1 + a), the first factor without cancellation
    a = torch.exp(-fall)
    return a, torch.sqrt(-torch.expm1(-fall) * (1 + a)) * torch.sigmoid(i + b_i) * v
