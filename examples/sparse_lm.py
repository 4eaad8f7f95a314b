"""A small language model of truly sparse layers, trained on its own text.

    python examples/sparse_lm.py [--steps N] [--vocab V] [--width D] [--hidden H] [--dtype f32|bf16]

Every token predicts the next one through an embedding, a residual block of two
sparse layers with GELU between them, and a projection to the vocabulary that
shares the embedding's table.  One training step runs, in order: embed, the
sparse forward, xent (the loss, without its logits), xent_grad, the sparse
backward, embed_grad (added to the table's gradient), clip_grad_norm, and plain
gradient descent; every `--rewire` steps each layer prunes and regrows a tenth
of its connections.  The text is a random Markov chain in which each token has
four likely successors, so a model that has learnt it has a loss near log 4.
"""

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

from spmm_row_sorted_gb300 import snack
from spmm_row_sorted_gb300 import workloads as wl


def chain_text(vocab: int, length: int, seed: int) -> np.ndarray:
    """Ids of a Markov chain: each token is followed by one of four fixed successors."""
    rng = np.random.default_rng(seed)
    after = rng.integers(0, vocab, (vocab, 4))
    pick = rng.integers(0, 4, length)
    ids = np.empty(length, dtype=np.int64)
    ids[0] = 0
    for i in range(1, length):
        ids[i] = after[ids[i - 1], pick[i]]
    return ids


class SparseLM:
    def __init__(self, vocab: int, width: int, hidden: int, density: float, batch: int, dtype: str = "f32", seed: int = 0):
        kind = torch.float32 if dtype == "f32" else torch.bfloat16
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.scale = vocab, math.sqrt(width)
        self.table = (torch.empty(vocab, width, device="cuda").normal_(generator=gen) / width).to(kind)

        def layer(out_f, in_f, k):
            lay = wl.make_layer(out_f, in_f, density=density, val_std=math.sqrt(1.0 / (density * in_f)), seed=seed + k)
            row, col, val = (torch.from_numpy(a).cuda() for a in (lay.row, lay.col, lay.val))
            return snack.SparseLinear(out_f, in_f, row, col, val.to(kind), torch.zeros(out_f, device="cuda"), max_batch=batch)

        self.up, self.down = layer(hidden, width, 1), layer(width, hidden, 2)

    def step(self, ids: torch.Tensor, targets: torch.Tensor, lr: float, max_norm: float) -> tuple:
        """One training step; returns (loss, gradient norm) as CUDA scalars."""
        x = snack.embed(ids, self.table, self.scale)
        h, pre = self.up.forward_gelu(x)
        y = x + self.down.forward(h)
        loss, state = snack.xent(y, self.table, targets)

        dy, dtable = snack.xent_grad(y, self.table, targets, state)
        dpre = self.down.grad_input_gelu(dy, pre)
        dw_down, db_down = self.down.grad_weight(h, dy)
        dx_up, dw_up, db_up = self.up.backward(x, dpre)
        snack.embed_grad(ids, dy + dx_up, self.vocab, self.scale, out=dtable, accumulate=True)

        grads = [dtable, dw_up, db_up, dw_down, db_down]
        norm = snack.clip_grad_norm(grads, max_norm)
        for param, grad in zip((self.table, self.up.val, self.up.bias, self.down.val, self.down.bias), grads):
            param.sub_((lr * grad.float()).to(param.dtype))
        return loss, norm

    def rewire(self, step: int, seed: int = 0) -> None:
        for k, layer in enumerate((self.up, self.down)):
            layer.restructure(layer.nnz // 10, seed + k, step)

    def close(self) -> None:
        self.up.close()
        self.down.close()


def train(steps: int = 400, vocab: int = 1000, width: int = 256, hidden: int = 1024, density: float = 0.05,
          batch: int = 1024, rewire: int = 100, lr: float = 1.5, max_norm: float = 1.0, dtype: str = "f32", seed: int = 0,
          report=None) -> list:
    """Train and return the loss of every step."""
    text = torch.from_numpy(chain_text(vocab, batch * 64 + 1, seed)).cuda()
    model = SparseLM(vocab, width, hidden, density, batch, dtype, seed)
    losses = []
    for i in range(steps):
        at = (i % 64) * batch
        loss, norm = model.step(text[at:at + batch], text[at + 1:at + batch + 1], lr, max_norm)
        losses.append(loss)
        if rewire and (i + 1) % rewire == 0 and i + 1 < steps:
            model.rewire(i)
        if report and (i % report == 0 or i + 1 == steps):
            print(f"step {i:5d}  loss {float(loss):.4f}  gradient norm {float(norm):.3f}", flush=True)
    out = [float(v) for v in losses]
    model.close()
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=400)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--batch", type=int, default=1024)
    ap.add_argument("--rewire", type=int, default=100)
    ap.add_argument("--lr", type=float, default=1.5)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    a = ap.parse_args()
    train(a.steps, a.vocab, a.width, a.hidden, batch=a.batch, rewire=a.rewire, lr=a.lr, dtype=a.dtype, report=20)
