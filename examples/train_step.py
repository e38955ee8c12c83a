"""A small recommendation model trained with the library's calls only (and torch's matrix products between them):

  ids -> pooled rows (TableBatchedEmbedding.forward) -> layer norm of each table's rows (LayerNorm)
      -> two dense layers -> click probability
  and back: dx of the layer norm is the embedding's grad_out (backward_update, row-wise Adagrad); the dense
  gradients are clipped by their global norm (GradNorm) and applied by DenseAdamW.

No call in a step synchronizes with the host.  Run: python examples/train_step.py [--states q8] [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bwd_tbe_fwd_gb300 import DenseAdamW, GradNorm, LayerNorm, TableBatchedEmbedding  # noqa: E402

D, E, BAGS, LOOKUPS, HIDDEN = [32, 64, 128, 32], [2000, 500, 3000, 100], 1024, 4, 64


class Model:
    def __init__(self, states: str = "f32", seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.g = g
        n = len(D) * BAGS * LOOKUPS
        self.tbe = TableBatchedEmbedding(D, E, BAGS, n, torch.float16, device=device)
        self.tables = (0.02 * (torch.rand(self.tbe.num_weights, generator=g) - 0.5)).half().to(device)
        self.state = torch.zeros(self.tbe.total_rows, device=device)
        self.offsets = torch.arange(0, n + 1, LOOKUPS, device=device)
        self.norm = LayerNorm(self.tbe.D, device=device)
        width = sum(D)
        shapes = [(width, HIDDEN), (HIDDEN, 1), (width,), (width,), (HIDDEN,), (1,)]  # w1 w2 | gain shift b1 b2
        self.params = [torch.randn(s, generator=g).mul_(s[0] ** -0.5) if len(s) == 2 else torch.zeros(s) for s in shapes]
        self.params[2].fill_(1.0)
        self.params = [p.to(device) for p in self.params]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.clip = GradNorm(self.grads)
        self.opt = DenseAdamW(self.params, self.grads, states, weight_decay=[0.01, 0.01, 0.0, 0.0, 0.0, 0.0])
        self.taste = [torch.randn(e, generator=g) for e in E]  # what the labels depend on

    def batch(self):
        """Ids, and clicks that the sum of the looked-up rows' tastes makes likely."""
        ids = [torch.randint(0, e, (BAGS, LOOKUPS), generator=self.g) for e in E]
        score = sum(t[i].sum(1) for t, i in zip(self.taste, ids))
        clicks = (torch.rand(BAGS, generator=self.g) < torch.sigmoid(score)).float()
        return torch.cat([i.reshape(-1) for i in ids]).to(self.offsets.device), clicks.to(self.offsets.device)

    def step(self, ids, clicks, lr: float):
        """One training step; returns the loss as a device scalar."""
        w1, w2, gain, shift, b1, b2 = self.params
        pooled = self.tbe.forward(self.tables, ids, self.offsets)
        y, mean, rstd = self.norm.forward(pooled, gain, shift)
        hidden = torch.relu(y @ w1 + b1)
        logit = (hidden @ w2 + b2).squeeze(1)
        loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, clicks)

        d_logit = ((torch.sigmoid(logit) - clicks) / BAGS)[:, None]
        d_hidden = (d_logit @ w2.T) * (hidden > 0)
        g1, g2, g_gain, g_shift, gb1, gb2 = self.grads
        torch.mm(y.T, d_hidden, out=g1)
        torch.mm(hidden.T, d_logit, out=g2)
        torch.sum(d_hidden, 0, out=gb1)
        torch.sum(d_logit, 0, out=gb2)
        dx, _, _ = self.norm.backward(d_hidden @ w1.T, pooled, mean, rstd, gain, dweight=g_gain, dbias=g_shift)
        self.tbe.backward_update(self.tables, self.state, ids, self.offsets, dx, optimizer="adagrad", lr=lr)
        self.opt.step(lr, clip=self.clip.compute(1.0))
        return loss


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--states", choices=("f32", "q8"), default="f32", help="AdamW's states: 32 or 8 bits")
    ap.add_argument("--steps", type=int, default=300)
    a = ap.parse_args()
    model = Model(a.states)
    losses = []
    for k in range(a.steps):
        losses.append(model.step(*model.batch(), lr=3e-3))
        if (k + 1) % 50 == 0:
            print(f"step {k + 1}: loss {float(torch.stack(losses[-50:]).mean()):.4f}")


if __name__ == "__main__":
    main()
