"""A small next-item model trained with the library's calls (and torch's matrix product between them): one table of items at
both ends.

  ids -> the table's rows (TokenEmbedding.forward) -> layer norm (LayerNorm) -> a dense layer with a residual
      -> softmax over the same table's rows (SoftmaxLoss), the next id of each sequence the target, padding ignored
  and back: the loss leaves the table's gradient, the lookup's gradient adds to it (accumulate), all gradients are clipped by
  their global norm (GradNorm) and applied to bf16 parameters with fp32 masters by DenseAdamW.

No call in a step synchronizes with the host.  Run: python examples/train_items.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from bwd_tbe_fwd_gb300 import DenseAdamW, GradNorm, LayerNorm, SoftmaxLoss, TokenEmbedding  # noqa: E402

ITEMS, WIDTH, SEQUENCES, LENGTH = 1000, 64, 64, 16
BF16 = torch.bfloat16


class Model:
    def __init__(self, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.g, self.device = g, device
        tokens = SEQUENCES * LENGTH
        self.lookup = TokenEmbedding(ITEMS, WIDTH, tokens, table_dtype=BF16, out_dtype=torch.float32, scale=WIDTH ** 0.5,
                                     device=device)
        self.norm = LayerNorm(WIDTH, x_dtype=torch.float32, y_dtype=BF16, weight_dtype=BF16, device=device)
        self.loss = SoftmaxLoss(ITEMS, WIDTH, tokens, dtype=BF16, device=device)
        table = torch.randn(ITEMS, WIDTH, generator=g) * WIDTH ** -0.5
        dense = torch.randn(WIDTH, WIDTH, generator=g) * WIDTH ** -0.5
        self.masters = [t.to(device) for t in (table, dense, torch.ones(WIDTH), torch.zeros(WIDTH))]
        self.params = [t.to(BF16) for t in self.masters]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.clip = GradNorm(self.grads)
        self.opt = DenseAdamW(self.params, self.grads, master=self.masters, weight_decay=[0.0, 0.01, 0.0, 0.0])
        self.follows = torch.randint(0, ITEMS, (ITEMS, 2), generator=g)  # what comes after an item

    def batch(self):
        """Ids and the ids that follow them, [SEQUENCES, LENGTH] each, the sequences' ends padded with -1."""
        ids = [torch.randint(0, ITEMS, (SEQUENCES,), generator=self.g)]
        for _ in range(LENGTH):
            ids.append(self.follows[ids[-1], torch.randint(0, 2, (SEQUENCES,), generator=self.g)])
        ids = torch.stack(ids, 1)
        ends = torch.randint(LENGTH // 2, LENGTH + 1, (SEQUENCES, 1), generator=self.g)
        past = torch.arange(LENGTH) >= ends
        pad = torch.full((SEQUENCES, LENGTH), -1)
        return (torch.where(past, pad, ids[:, :-1]).to(self.device), torch.where(past, pad, ids[:, 1:]).to(self.device))

    def step(self, ids, targets, lr: float):
        """One training step; returns {mean loss, 1 / tokens that count} on the device."""
        table, dense, gain, shift = self.params
        g_table, g_dense, g_gain, g_shift = self.grads
        rows = self.lookup.forward(table, ids).view(-1, WIDTH)
        y, mean, rstd = self.norm.forward(rows, gain, shift)
        hidden = torch.addmm(y, y, dense)
        targets = targets.view(-1)
        _, lse, result = self.loss.forward(hidden, table, targets)

        d_hidden, _ = self.loss.backward(hidden, table, targets, lse, mean=result, dweight=g_table)
        torch.mm(y.T, d_hidden, out=g_dense)
        d_y = torch.addmm(d_hidden, d_hidden, dense.T)
        d_rows, _, _ = self.norm.backward(d_y, rows, mean, rstd, gain, dweight=g_gain, dbias=g_shift)
        self.lookup.backward(d_rows, ids, grad=g_table, accumulate=True)
        self.opt.step(lr, clip=self.clip.compute(1.0))
        return result


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=400)
    a = ap.parse_args()
    model = Model()
    losses = []
    for k in range(a.steps):
        losses.append(model.step(*model.batch(), lr=3e-3)[0])
        if (k + 1) % 50 == 0:
            print(f"step {k + 1}: loss {float(torch.stack(losses[-50:]).mean()):.4f}")


if __name__ == "__main__":
    main()
