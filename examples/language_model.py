"""A small recurrent language model, trained with the library's own operators.

    tokens -> embedding -> [norm -> input projection -> recurrence -> gated,
    scaled residual (-> norm -> gated feed-forward -> dropout -> residual)] x blocks
    -> norm -> cross entropy over the vocabulary

The recurrence is the diagonal GRU by Newton iterations, or (cell="linear") the gated
linear recurrence; mlp gives every block a feed-forward part of that many times the
width.  The embedding weight is also the vocabulary's (its gradient comes from both
ends).  The gate and the gradients of the two projections are plain matrix
products.  Run it to train on synthetic text, a Markov chain over the vocabulary:

    python examples/language_model.py --steps 200
    python examples/language_model.py --steps 200 --cell linear --mlp 4 --dropout 0.1
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nonlinear_rnn_gb300 as nr  # noqa: E402

IGNORE = -100


class LanguageModel:
    """Weights by name; loss() and gradients() of a batch of token sequences."""

    def __init__(self, vocab: int, d: int, blocks: int, dtype=torch.bfloat16, K: int = 3, seed: int = 0,
                 cell: str = "gru", mlp: int = 0, p: float = 0.0):
        self.vocab, self.d, self.blocks, self.dtype, self.K = vocab, d, blocks, dtype, K
        self.cell, self.mlp, self.p = cell, mlp, p
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std
        ones = torch.ones(d, device="cuda")
        self.embed_scale, self.logit_scale = math.sqrt(d), 1.0
        w = {"embed": normal(vocab, d, std=1 / math.sqrt(d)).to(dtype)}
        for b in range(blocks):
            w[f"{b}.W_x"] = normal(3 * d, d, std=1 / math.sqrt(d)).to(dtype)
            w[f"{b}.W_gate"] = normal(d, d, std=1 / math.sqrt(d)).to(dtype)
            if cell == "gru":
                w[f"{b}.cell"] = torch.rand(6, d, generator=g, device="cuda") * 2 - 1
            else:   # rows log rate (decays of 0.9 to 0.99 at an open gate), b_a, b_i
                w[f"{b}.cell"] = normal(3, d, std=0.3)
                w[f"{b}.cell"][0] = (-(torch.rand(d, generator=g, device="cuda") * 0.09 + 0.9).log()).log()
            w[f"{b}.w_pre"], w[f"{b}.w_post"] = ones.clone(), ones.clone()
            w[f"{b}.scale"] = ones / math.sqrt(2 * blocks)
            if mlp:
                w[f"{b}.w_mlp"] = ones.clone()
                w[f"{b}.W_in"] = normal(2 * mlp * d, d, std=1 / math.sqrt(d)).to(dtype)
                w[f"{b}.W_out"] = normal(d, mlp * d, std=1 / math.sqrt(2 * blocks * mlp * d)).to(dtype)
        w["w_out"] = ones.clone()
        self.weights = w

    def _pre(self, b: int) -> torch.Tensor:
        """The norm weight in front of block b, or of the vocabulary after the last."""
        return self.weights[f"{b}.w_pre"] if b < self.blocks else self.weights["w_out"]

    def _rec(self, b: int) -> torch.Tensor:
        """The linear recurrence's parameters: rate, b_a, b_i."""
        c = self.weights[f"{b}.cell"]
        return torch.cat([c[:1].exp(), c[1:]])

    def _recurrence(self, b: int, P: torch.Tensor) -> torch.Tensor:
        if self.cell == "gru":
            return nr.newton_forward(P, self.weights[f"{b}.cell"], K=self.K, check=False)[0]
        return nr.linear_recurrence(P, self._rec(b))[0]

    def forward(self, tokens: torch.Tensor, step: int | None = None):
        """Last normalised states (B, T, d) and what the backward needs.  step: the
        training step, which dropout takes its mask from (None: no dropout)."""
        w = self.weights
        x = nr.embedding(tokens, w["embed"], scale=self.embed_scale)
        first, u = x, nr.block_norm(x, w_pre=self._pre(0))[1]
        kept = []
        for b in range(self.blocks):
            P = nr.input_projection(u, w[f"{b}.W_x"])
            gate = u @ w[f"{b}.W_gate"].T
            H = self._recurrence(b, P)
            w_next = w[f"{b}.w_mlp"] if self.mlp else self._pre(b + 1)
            x, v = nr.block_norm(x, h=H, gate=gate, w_post=w[f"{b}.w_post"], scale=w[f"{b}.scale"], w_pre=w_next)
            feed = None
            if self.mlp:
                y, inner = nr.gated_mlp(v, w[f"{b}.W_in"], w[f"{b}.W_out"], keep=True)
                x2 = nr.dropout(y, 0.0 if step is None else self.p, step or 0, offset=b, residual=x)
                feed, v = (v, inner, x2), nr.block_norm(x2, w_pre=self._pre(b + 1))[1]
            kept.append((u, P, gate, H, x, feed))
            x, u = (feed[2] if self.mlp else x), v
        return u, (first, kept)

    def step(self, tokens: torch.Tensor, states: list | None = None):
        """One token per slot, tokens (slots): the logits (slots, vocab) and the states
        that the next step takes (None: an empty history).  The linear cell only."""
        w = self.weights
        x = nr.embedding(tokens, w["embed"], scale=self.embed_scale)
        u, new = nr.block_norm(x, w_pre=self._pre(0))[1], []
        for b in range(self.blocks):
            P = nr.input_projection(u, w[f"{b}.W_x"])
            gate = u @ w[f"{b}.W_gate"].T
            h, state = nr.linear_recurrence_step(self._rec(b), None if states is None else states[b], P)
            new.append(state)
            w_next = w[f"{b}.w_mlp"] if self.mlp else self._pre(b + 1)
            x, u = nr.block_norm(x, h=h, gate=gate, w_post=w[f"{b}.w_post"], scale=w[f"{b}.scale"], w_pre=w_next)
            if self.mlp:
                x = x + nr.gated_mlp(u, w[f"{b}.W_in"], w[f"{b}.W_out"])
                u = nr.block_norm(x, w_pre=self._pre(b + 1))[1]
        return self.logit_scale * u.float() @ w["embed"].float().T, new

    def loss(self, tokens: torch.Tensor, targets: torch.Tensor, step: int | None = None) -> torch.Tensor:
        """Mean loss over the targets that are not IGNORE."""
        u, _ = self.forward(tokens, step)
        loss, _ = nr.vocab_loss(u, self.weights["embed"], targets, logit_scale=self.logit_scale, ignore_index=IGNORE)
        return loss.sum() / (targets != IGNORE).sum()

    def gradients(self, tokens: torch.Tensor, targets: torch.Tensor, step: int | None = None):
        """(mean loss, gradients by the weights' names)."""
        w, g = self.weights, {}
        u, (first, kept) = self.forward(tokens, step)
        count = (targets != IGNORE).sum()
        loss, lse = nr.vocab_loss(u, w["embed"], targets, logit_scale=self.logit_scale, ignore_index=IGNORE)
        g_loss = (torch.ones_like(loss) / count).contiguous()
        gu, g["embed"] = nr.vocab_loss_backward(u, w["embed"], targets, lse, g_loss,
                                                logit_scale=self.logit_scale, ignore_index=IGNORE)
        gx = None
        for b in reversed(range(self.blocks)):
            u, P, gate, H, x, feed = kept[b]
            w_next, name = self._pre(b + 1), "w_out" if b + 1 == self.blocks else f"{b + 1}.w_pre"
            if self.mlp:
                v, inner, x2 = feed
                r = nr.block_norm_backward(x2, w_pre=w_next, g_x=gx, g_u=gu)
                g[name], gx = r.gw_pre, r.gx
                gy = nr.dropout(gx, 0.0 if step is None else self.p, step or 0, offset=b)
                gu, g[f"{b}.W_in"], g[f"{b}.W_out"] = nr.gated_mlp_backward(v, w[f"{b}.W_in"], w[f"{b}.W_out"], inner, gy)
                w_next, name = w[f"{b}.w_mlp"], f"{b}.w_mlp"
            r = nr.block_norm_backward(x, h=H, gate=gate, w_post=w[f"{b}.w_post"], scale=w[f"{b}.scale"],
                                       w_pre=w_next, g_x=gx, g_u=gu)
            g[name] = r.gw_pre
            g[f"{b}.w_post"], g[f"{b}.scale"], gx = r.gw_post, r.g_scale, r.gx
            if self.cell == "gru":
                gP, g[f"{b}.cell"] = nr.newton_backward(P, w[f"{b}.cell"], H, r.gh)
            else:
                gP, gc, _ = nr.linear_recurrence_backward(P, self._rec(b), H, r.gh)
                gc[0] *= w[f"{b}.cell"][0].exp()
                g[f"{b}.cell"] = gc
            rows = u.reshape(-1, self.d)
            g[f"{b}.W_x"] = gP.reshape(-1, 3 * self.d).T @ rows
            g[f"{b}.W_gate"] = r.g_gate.reshape(-1, self.d).T @ rows
            gu = gP @ w[f"{b}.W_x"] + r.g_gate @ w[f"{b}.W_gate"]
        r = nr.block_norm_backward(first, w_pre=self._pre(0), g_u=gu)
        g["0.w_pre"] = r.gw_pre
        # the residual stream and the first norm both lead back to the embedding
        nr.embedding_backward(tokens, r.gx + gx, self.vocab, scale=self.embed_scale,
                              out=g["embed"], accumulate=True)
        return loss.sum() / count, g


class Adam:
    def __init__(self, weights: dict, lr: float = 2e-3):
        self.master = {k: v.float() for k, v in weights.items()}
        self.m = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.v = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.t, self.lr = 0, lr

    def step(self, weights: dict, grads: dict) -> None:
        self.t += 1
        for k, g in grads.items():
            g = g.float()
            self.m[k].mul_(0.9).add_(g, alpha=0.1)
            self.v[k].mul_(0.99).addcmul_(g, g, value=0.01)
            m, v = self.m[k] / (1 - 0.9 ** self.t), self.v[k] / (1 - 0.99 ** self.t)
            self.master[k] -= self.lr * m / (v.sqrt() + 1e-8)
            weights[k].copy_(self.master[k])


def markov_batch(g: torch.Generator, table: torch.Tensor, B: int, T: int) -> torch.Tensor:
    """B sequences of T + 1 tokens: each token has a few likely successors (table)."""
    out = torch.empty(B, T + 1, dtype=torch.int64, device="cuda")
    out[:, 0] = torch.randint(0, table.shape[0], (B,), generator=g, device="cuda")
    pick = torch.randint(0, table.shape[1], (B, T), generator=g, device="cuda")
    for t in range(T):
        out[:, t + 1] = table[out[:, t], pick[:, t]]
    return out


def train(steps: int, vocab: int = 2000, d: int = 256, blocks: int = 2, B: int = 16, T: int = 256,
          dtype=torch.bfloat16, seed: int = 0, report=None, cell: str = "gru", mlp: int = 0,
          p: float = 0.0) -> list[float]:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randint(0, vocab, (vocab, 4), generator=g, device="cuda")
    model = LanguageModel(vocab, d, blocks, dtype=dtype, seed=seed, cell=cell, mlp=mlp, p=p)
    adam = Adam(model.weights)
    losses = []
    for i in range(steps):
        tokens = markov_batch(g, table, B, T)
        targets = tokens[:, 1:].clone()
        targets[:, :1] = IGNORE   # the first token has nothing before it to go by
        loss, grads = model.gradients(tokens[:, :-1].contiguous(), targets, step=i)
        adam.step(model.weights, grads)
        losses.append(float(loss))
        if report is not None:
            report(i, losses[-1])
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--vocab", type=int, default=2000)
    ap.add_argument("--d", type=int, default=256)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--cell", choices=("gru", "linear"), default="gru")
    ap.add_argument("--mlp", type=int, default=0, help="inner width of the feed-forward part over d (0: none)")
    ap.add_argument("--dropout", type=float, default=0.0, help="of the feed-forward part's output")
    a = ap.parse_args()

    def report(i, loss):
        if i % 20 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {loss:.3f}  (uniform {math.log(a.vocab):.3f}, floor {math.log(4):.3f})", flush=True)
    train(a.steps, a.vocab, a.d, a.blocks, report=report, cell=a.cell, mlp=a.mlp, p=a.dropout)
