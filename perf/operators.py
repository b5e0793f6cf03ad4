"""The operators of a language model around the recurrent layer, as cases to run.

Three operators and their gradients: the embedding lookup that feeds the first
block, the norms around a block with its gate and residual scale, and the
cross entropy over the vocabulary that ends the model.  ``run`` computes a case
with the library's kernels (``own``) or in plain fp32 torch operations, and
``exact`` gives the same outputs from the definitions in float64.

Widths, row counts and packs follow the recurrent layer's own workloads (d_h
64, 256, 512, 1024; 16 x 16384 and 262144 tokens); vocabularies are 32768 and
65536 rows, and sizes that no tile divides."""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
IGNORE = -100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
#: rows x vocabulary x width of the largest listed loss, which no drawn one passes
MOST_LOSS = 16384 * 65536 * 1024
#: elements of the widest listed activations
MOST_ELEMENTS = 262144 * 1024


def listed():
    return [
        # one decode step: the ids of 16 slots to their embedding rows
        {"name": "embed_step", "op": "embed", "way": "forward", "type": "bf16", "n": 16, "v": 32768, "d": 1024, "pad": 0.0},
        # the ragged pack of 262144 tokens, fp32
        {"name": "embed_pack_f32", "op": "embed", "way": "forward", "type": "f32", "n": 262144, "v": 65536, "d": 512, "pad": 0.02},
        # the gradient of an odd batch with padding: no size divides a tile or a 16-byte load
        {"name": "embed_grad_odd_f32", "op": "embed", "way": "backward", "type": "f32", "n": 30001, "v": 50021, "d": 250, "pad": 0.1},
        # the gradient of a training batch of 16 rows of 16384 tokens
        {"name": "embed_grad_bf16", "op": "embed", "way": "backward", "type": "bf16", "n": 262144, "v": 65536, "d": 1024, "pad": 0.0},
        # the norms of one decode step of 8 slots
        {"name": "norm_step", "op": "norm", "way": "forward", "type": "bf16", "n": 8, "d": 1024, "gate": True},
        # the norms of a training batch of 16 rows of 16384 tokens
        {"name": "norm_bf16", "op": "norm", "way": "forward", "type": "bf16", "n": 262144, "d": 1024, "gate": True},
        # the gradient of the 8 x 4096 workload's norms, fp32
        {"name": "norm_grad_f32", "op": "norm", "way": "backward", "type": "f32", "n": 32768, "d": 256, "gate": True},
        # the gradient of an odd width, without a gate
        {"name": "norm_grad_odd_bf16", "op": "norm", "way": "backward", "type": "bf16", "n": 65537, "d": 515, "gate": False},
        # scoring the next token of 4 slots over an odd vocabulary
        {"name": "loss_step", "op": "loss", "way": "forward", "type": "bf16", "n": 4, "v": 50021, "d": 1024, "ignored": 0.0},
        # a training step of an odd fp32 batch, three rows in ten ignored
        {"name": "loss_odd_f32", "op": "loss", "way": "train", "type": "f32", "n": 3001, "v": 10007, "d": 250, "ignored": 0.3},
        # a training step of 4096 tokens with some padding
        {"name": "loss_bf16", "op": "loss", "way": "train", "type": "bf16", "n": 4096, "v": 32768, "d": 512, "ignored": 0.05},
        # one 16384-token row of the widest workload over a large vocabulary
        {"name": "loss_large_bf16", "op": "loss", "way": "train", "type": "bf16", "n": 16384, "v": 65536, "d": 1024, "ignored": 0.0},
    ]


def spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def width(rng, low, high):
    """A width: one in two divides by 64, as layers' widths do; the others fall anywhere."""
    d = spread(rng, low, high)
    return d if rng.random() < 0.5 else max(low, d // 64 * 64)


def draw(rng):
    kind = rng.choice(("embed", "norm", "loss"))
    case = {"op": kind, "type": rng.choice(("bf16", "f32"))}
    if kind == "loss":
        d, v = width(rng, 64, 1024), spread(rng, 1000, 65536)
        n = spread(rng, 1, min(16384, MOST_LOSS // (d * v)))
        return {**case, "way": rng.choice(("forward", "train")), "n": n, "v": v, "d": d, "ignored": rng.choice((0.0, 0.1, 0.5))}
    d = width(rng, 64, 1024)
    n = spread(rng, 1, min(262144, MOST_ELEMENTS // d // (1 if case["type"] == "bf16" else 2)))
    case.update(way=rng.choice(("forward", "backward")), n=n, d=d)
    if kind == "norm":
        return {**case, "gate": rng.random() < 0.7}
    return {**case, "v": spread(rng, 1000, 65536), "pad": rng.choice((0.0, 0.05))}


def token_ids(g, n, v):
    """Ids whose frequency falls as one over their rank, as words' do."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (float(v) ** u).long().clamp_(1, v) - 1


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    n, d, t = case["n"], case["d"], TYPES[case["type"]]

    def normal(*shape, std=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = {"op": case["op"], "way": case["way"]}
    if case["op"] == "embed":
        v = case["v"]
        ids = token_ids(g, n, v)
        s["padding_idx"] = v - 1
        if case["pad"]:
            ids[torch.rand(n, generator=g, device="cuda") < case["pad"]] = v - 1
        s.update(ids=ids, v=v, scale=math.sqrt(d))
        if case["way"] == "forward":
            s["W"] = normal(v, d, std=1 / math.sqrt(d))
        else:
            s["g"] = normal(n, d, std=0.1)
    elif case["op"] == "norm":
        f32 = torch.float32
        s["h"] = normal(n, d, std=0.4)                 # a block's states, |h| < 1 mostly
        s["gate"] = normal(n, d) if case["gate"] else None
        s["w_post"] = 1 + normal(d, std=0.1, dtype=f32)
        s["scale"] = 0.5 + normal(d, std=0.1, dtype=f32)
        s["w_pre"] = 1 + normal(d, std=0.1, dtype=f32)
        if case["way"] == "forward":
            s["x"] = normal(n, d, std=2.0)
        else:
            s["x_out"] = normal(n, d, std=2.0)
            s["g_x"] = normal(n, d, std=0.1)
            s["g_u"] = normal(n, d, std=0.1)
    else:
        v = case["v"]
        s["x"] = normal(n, d)
        s["W"] = normal(v, d, std=2 / math.sqrt(d))
        t_ids = token_ids(g, n, v)
        # a model that has learnt something: some rows lean towards their target
        lean = torch.rand(n, 1, generator=g, device="cuda") * 1.5
        s["x"] = (s["x"].float() + lean * s["W"][t_ids].float()).to(t)
        if case["ignored"]:
            t_ids[torch.rand(n, generator=g, device="cuda") < case["ignored"]] = IGNORE
        s["targets"] = t_ids
        s["g_loss"] = torch.full((n,), 1.0 / n, device="cuda")
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import nonlinear_rnn_gb300 as nr

    if s["op"] == "embed":
        if s["way"] == "forward":
            return {"rows": nr.embedding(s["ids"], s["W"], scale=s["scale"], padding_idx=s["padding_idx"])}
        return {"gW": nr.embedding_backward(s["ids"], s["g"], s["v"], scale=s["scale"], padding_idx=s["padding_idx"])}
    if s["op"] == "norm":
        if s["way"] == "forward":
            x_out, u = nr.block_norm(s["x"], h=s["h"], gate=s["gate"], w_post=s["w_post"], scale=s["scale"], w_pre=s["w_pre"], eps=EPS)
            return {"x_out": x_out, "u": u}
        r = nr.block_norm_backward(s["x_out"], h=s["h"], gate=s["gate"], w_post=s["w_post"], scale=s["scale"], w_pre=s["w_pre"], g_x=s["g_x"], g_u=s["g_u"], eps=EPS)
        return r._asdict()
    loss, lse = nr.vocab_loss(s["x"], s["W"], s["targets"], ignore_index=IGNORE)
    if s["way"] == "forward":
        return {"loss": loss, "lse": lse}
    gx, gW = nr.vocab_loss_backward(s["x"], s["W"], s["targets"], lse, s["g_loss"], ignore_index=IGNORE)
    return {"loss": loss, "lse": lse, "gx": gx, "gW": gW}


def run_plain(s):
    if s["op"] == "embed":
        ids = s["ids"]
        kept = (ids != s["padding_idx"])[:, None]
        if s["way"] == "forward":
            rows = s["W"][ids].float() * s["scale"]
            return {"rows": torch.where(kept, rows, 0.0).to(s["W"].dtype)}
        g = torch.where(kept, s["g"].float(), 0.0) * s["scale"]
        gW = torch.zeros(s["v"], g.shape[1], device=g.device).index_add_(0, ids, g)
        return {"gW": gW.to(s["g"].dtype)}
    if s["op"] == "norm":
        return plain_norm(s) if s["way"] == "forward" else plain_norm_backward(s)
    t = s["x"].dtype
    kept = s["targets"] != IGNORE
    at = torch.where(kept, s["targets"], 0)[:, None]
    x, W = torch.where(kept[:, None], s["x"].float(), 0.0), s["W"].float()
    z = x @ W.T
    most = z.max(1, keepdim=True).values
    e = (z - most).exp()
    total = e.sum(1, keepdim=True)
    lse = most + total.log()
    loss = torch.where(kept, (lse - z.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": torch.where(kept, lse[:, 0], 0.0)}
    if s["way"] == "train":
        del z
        gz = e / total
        del e
        gz.scatter_add_(1, at, torch.full_like(lse, -1.0))
        gz *= torch.where(kept, s["g_loss"], 0.0)[:, None]
        out["gx"] = (gz @ W).to(t)
        out["gW"] = (gz.T @ x).to(t)
    return out


def plain_norm(s):
    t = s["x"].dtype
    x, h = s["x"].float(), s["h"].float()
    y = h * (1 / ((h * h).mean(1, keepdim=True) + EPS).sqrt()) * s["w_post"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        y = y * (gate / (1 + (-gate).exp()))
    x_out = x + s["scale"] * y
    u = x_out * (1 / ((x_out * x_out).mean(1, keepdim=True) + EPS).sqrt()) * s["w_pre"]
    return {"x_out": x_out.to(t), "u": u.to(t)}


def plain_norm_backward(s):
    t = s["x_out"].dtype
    x, h, g_x, g_u = (s[k].float() for k in ("x_out", "h", "g_x", "g_u"))
    r = 1 / ((x * x).mean(1, keepdim=True) + EPS).sqrt()
    xn = x * r
    a = g_u * s["w_pre"]
    gx = g_x + r * (a - xn * (a * xn).mean(1, keepdim=True))
    q = 1 / ((h * h).mean(1, keepdim=True) + EPS).sqrt()
    hn = h * q
    gate_of = dgate = None
    if s["gate"] is not None:
        gate = s["gate"].float()
        sig = 1 / (1 + (-gate).exp())
        gate_of, dgate = gate * sig, sig * (1 + gate * (1 - sig))
    y = hn * s["w_post"] if gate_of is None else hn * s["w_post"] * gate_of
    gy = gx * s["scale"]
    gn = gy if gate_of is None else gy * gate_of
    b = gn * s["w_post"]
    gh = q * (b - hn * (b * hn).mean(1, keepdim=True))
    return {
        "gx": gx.to(t),
        "gh": gh.to(t),
        "g_gate": None if dgate is None else (gy * hn * s["w_post"] * dgate).to(t),
        "gw_post": (gn * hn).sum(0),
        "g_scale": (gx * y).sum(0),
        "gw_pre": (g_u * xn).sum(0),
    }


def distinct(n, v):
    """The expected number of distinct ids among n of token_ids()."""
    k = np.arange(1, v + 1, dtype=np.float64)
    p = np.log1p(1 / k) / math.log(v) if v > 1 else np.ones(1)
    p[-1] = max(0.0, 1 - p[:-1].sum())
    return float((1 - np.exp(n * np.log1p(-np.minimum(p, 1 - 1e-12)))).sum())


def work(case):
    n, d = case["n"], case["d"]
    es = 2 if case["type"] == "bf16" else 4
    if case["op"] == "embed":
        rows = distinct(n, case["v"]) if case["way"] == "forward" else case["v"]
        return {"bytes": 8 * n + es * d * (n + rows), "flops": n * d}
    if case["op"] == "norm":
        gate = 1 if case["gate"] else 0
        if case["way"] == "forward":      # x, h and the gate in, x_out and u out
            return {"bytes": es * n * d * (4 + gate) + 12 * d, "flops": n * d * (10 + 5 * gate)}
        # x_out, h, the gate, g_x and g_u in; gx, gh and g_gate out
        return {"bytes": es * n * d * (6 + 2 * gate) + 24 * d, "flops": n * d * (30 + 10 * gate)}
    v, kept = case["v"], case["n"] * (1 - case["ignored"])
    if case["way"] == "forward":
        return {"bytes": es * d * (n + v) + 16 * n, "flops": 2 * kept * v * d}
    # forward, the logits once more for the gradient (they are not kept), and the two products of the gradient
    return {"bytes": 2 * es * d * (n + v) + 24 * n, "flops": 8 * kept * v * d}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "embed":
        dead = s["ids"] == s["padding_idx"]
        if case["way"] == "forward":
            rows = torch.index_select(s["W"], 0, s["ids"]).to(f64).mul_(s["scale"])
            return {"rows": rows.masked_fill_(dead[:, None], 0)}
        gW = torch.zeros(s["v"], case["d"], device="cuda", dtype=f64)
        for i in range(0, case["n"], 65536):
            live = ~dead[i:i + 65536]
            gW.index_add_(0, s["ids"][i:i + 65536][live], s["g"][i:i + 65536][live].to(f64))
        return {"gW": gW.mul_(s["scale"])}
    if case["op"] == "norm":
        return exact_norm(s, case)
    if 8 * case["n"] * case["v"] * case["d"] > 1.1e13:   # about 20 s of fp64
        return None
    n = case["n"]
    W = s["W"].to(f64)
    gW = torch.zeros_like(W) if case["way"] == "train" else None
    loss, lse = torch.zeros(n, device="cuda", dtype=f64), torch.zeros(n, device="cuda", dtype=f64)
    gx = torch.zeros(n, case["d"], device="cuda", dtype=f64)
    live = torch.nonzero(s["targets"] != IGNORE)[:, 0]
    for at in live.split(2048):
        x, t = s["x"][at].to(f64), s["targets"][at]
        logits = torch.matmul(x, W.t())
        lse[at] = torch.logsumexp(logits, 1)
        loss[at] = lse[at] - (x * W[t]).sum(1)
        if gW is not None:
            gl = torch.softmax(logits, 1)
            gl[torch.arange(t.numel(), device="cuda"), t] -= 1
            gl *= s["g_loss"][at].to(f64)[:, None]
            gx[at] = torch.matmul(gl, W)
            gW.addmm_(gl.t(), x)
    return {"loss": loss, "lse": lse} if gW is None else {"loss": loss, "lse": lse, "gx": gx, "gW": gW}


def exact_norm(s, case):
    """The norms in float64, rows in turn; the gradients by torch's differentiation of the forward formula."""
    f64, n, d = torch.float64, case["n"], case["d"]
    weights = [s[k].to(f64).requires_grad_(case["way"] == "backward") for k in ("w_post", "scale", "w_pre")]
    parts, sums = [], None

    def rms(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)

    for i in range(0, n, 32768):
        rows = {k: s[k][i:i + 32768].to(f64) for k in ("x", "x_out", "h", "gate", "g_x", "g_u") if s.get(k) is not None}
        y = rms(rows["h"].requires_grad_(case["way"] == "backward")) * weights[0]
        if "gate" in rows:
            rows["gate"].requires_grad_(case["way"] == "backward")
            y = y * torch.nn.functional.silu(y.new_tensor(1.0) * rows["gate"])
        if case["way"] == "forward":
            x_out = rows["x"] + weights[1] * y
            parts.append((x_out, rms(x_out) * weights[2]))
            continue
        # the stored x_out stands for x + scale y: its gradient goes on to both
        x_out = rows["x_out"].requires_grad_(True)
        gx, gw_pre = torch.autograd.grad([x_out * 1.0, rms(x_out) * weights[2]], [x_out, weights[2]], [rows["g_x"], rows["g_u"]])
        wanted = [rows["h"], weights[0], weights[1]] + ([rows["gate"]] if "gate" in rows else [])
        gh, gw_post, g_scale, *g_gate = torch.autograd.grad(weights[1] * y, wanted, gx)
        parts.append((gx, gh, *g_gate))
        add = torch.stack([gw_post, g_scale, gw_pre])
        sums = add if sums is None else sums + add
    cat = [torch.cat(c).detach() for c in zip(*parts)]
    if case["way"] == "forward":
        return {"x_out": cat[0], "u": cat[1]}
    return {"gx": cat[0], "gh": cat[1], "g_gate": cat[2] if len(cat) > 2 else None,
            "gw_post": sums[0].detach(), "g_scale": sums[1].detach(), "gw_pre": sums[2].detach()}
