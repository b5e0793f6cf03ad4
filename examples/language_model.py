"""A small recurrent language model, trained with the library's own operators.

    tokens -> embedding -> [norm -> input projection -> recurrence -> gated,
    scaled residual] x blocks -> norm -> cross entropy over the vocabulary

The embedding weight is also the vocabulary's (its gradient comes from both
ends).  The gate and the gradients of the two projections are plain matrix
products.  Run it to train on synthetic text, a Markov chain over the vocabulary:

    python examples/language_model.py --steps 200
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

    def __init__(self, vocab: int, d: int, blocks: int, dtype=torch.bfloat16, K: int = 3, seed: int = 0):
        self.vocab, self.d, self.blocks, self.dtype, self.K = vocab, d, blocks, dtype, K
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
            w[f"{b}.cell"] = torch.rand(6, d, generator=g, device="cuda") * 2 - 1
            w[f"{b}.w_pre"], w[f"{b}.w_post"] = ones.clone(), ones.clone()
            w[f"{b}.scale"] = ones / math.sqrt(2 * blocks)
        w["w_out"] = ones.clone()
        self.weights = w

    def _pre(self, b: int) -> torch.Tensor:
        """The norm weight in front of block b, or of the vocabulary after the last."""
        return self.weights[f"{b}.w_pre"] if b < self.blocks else self.weights["w_out"]

    def forward(self, tokens: torch.Tensor):
        """Last normalised states (B, T, d) and what the backward needs."""
        w = self.weights
        x = nr.embedding(tokens, w["embed"], scale=self.embed_scale)
        first, u = x, nr.block_norm(x, w_pre=self._pre(0))[1]
        kept = []
        for b in range(self.blocks):
            P = nr.input_projection(u, w[f"{b}.W_x"])
            gate = u @ w[f"{b}.W_gate"].T
            H, _ = nr.newton_forward(P, w[f"{b}.cell"], K=self.K, check=False)
            x, v = nr.block_norm(x, h=H, gate=gate, w_post=w[f"{b}.w_post"], scale=w[f"{b}.scale"],
                                 w_pre=self._pre(b + 1))
            kept.append((u, P, gate, H, x))
            u = v
        return u, (first, kept)

    def loss(self, tokens: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        """Mean loss over the targets that are not IGNORE."""
        u, _ = self.forward(tokens)
        loss, _ = nr.vocab_loss(u, self.weights["embed"], targets, logit_scale=self.logit_scale, ignore_index=IGNORE)
        return loss.sum() / (targets != IGNORE).sum()

    def gradients(self, tokens: torch.Tensor, targets: torch.Tensor):
        """(mean loss, gradients by the weights' names)."""
        w, g = self.weights, {}
        u, (first, kept) = self.forward(tokens)
        count = (targets != IGNORE).sum()
        loss, lse = nr.vocab_loss(u, w["embed"], targets, logit_scale=self.logit_scale, ignore_index=IGNORE)
        g_loss = (torch.ones_like(loss) / count).contiguous()
        gu, g["embed"] = nr.vocab_loss_backward(u, w["embed"], targets, lse, g_loss,
                                                logit_scale=self.logit_scale, ignore_index=IGNORE)
        gx = None
        for b in reversed(range(self.blocks)):
            u, P, gate, H, x = kept[b]
            r = nr.block_norm_backward(x, h=H, gate=gate, w_post=w[f"{b}.w_post"], scale=w[f"{b}.scale"],
                                       w_pre=self._pre(b + 1), g_x=gx, g_u=gu)
            g["w_out" if b + 1 == self.blocks else f"{b + 1}.w_pre"] = r.gw_pre
            g[f"{b}.w_post"], g[f"{b}.scale"], gx = r.gw_post, r.g_scale, r.gx
            gP, g[f"{b}.cell"] = nr.newton_backward(P, w[f"{b}.cell"], H, r.gh)
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
          dtype=torch.bfloat16, seed: int = 0, report=None) -> list[float]:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    table = torch.randint(0, vocab, (vocab, 4), generator=g, device="cuda")
    model = LanguageModel(vocab, d, blocks, dtype=dtype, seed=seed)
    adam = Adam(model.weights)
    losses = []
    for i in range(steps):
        tokens = markov_batch(g, table, B, T)
        targets = tokens[:, 1:].clone()
        targets[:, :1] = IGNORE   # the first token has nothing before it to go by
        loss, grads = model.gradients(tokens[:, :-1].contiguous(), targets)
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
    a = ap.parse_args()

    def report(i, loss):
        if i % 20 == 0 or i + 1 == a.steps:
            print(f"step {i:4d}  loss {loss:.3f}  (uniform {math.log(a.vocab):.3f}, floor {math.log(4):.3f})", flush=True)
    train(a.steps, a.vocab, a.d, a.blocks, report=report)
