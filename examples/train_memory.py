"""Trains a small hashed N-gram memory with the library's training calls.

    python examples/train_memory.py [--steps 40] [--tokens 8192]

One step, all of it on the current stream and without a host synchronisation:

  x     = pg.embed(tokens)                          token embedding, scaled
  e, y  = pg.gather_project_gate(tokens, x)         lookup, W_V and the scalar gate: y = x + g e W^T
  dy    = gradient of the loss at y
  dW    = g dy^T e,  de = g dy W                    plain matrix products
  dE    = pg.embed_grad(tokens, dy)                 the embedding's gradient (x enters y directly)
  rows, dT = pg.lookup_grad(tokens, de)             the table's gradient, distinct rows only
  O     = pg.orthogonalize(momentum of dW)          the projection's update

The loss is the squared distance to the outputs of a teacher of the same shape (random
embedding, table and projection), so it can be driven towards zero.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hashed_head_gram_gb300 import pg, workloads as W  # noqa: E402


class Memory:
    """fp32 master weights of the embedding, the table and W_V, with the bf16 copies that the
    lookup and the projection read."""

    def __init__(self, spec, vocab, d, seed, device, std):
        gen = torch.Generator(device=device).manual_seed(seed)
        rows, _, self.din = pg.table_geometry(pg.table_desc(spec, vocab))
        self.desc = pg.table_desc(spec, vocab)
        self.vocab, self.d, self.scale, self.g = vocab, d, float(d) ** 0.5, 0.5
        self.E = torch.randn(vocab, d, generator=gen, device=device) * std / self.scale
        self.T = torch.randn(rows + 1, spec.r, generator=gen, device=device) * std  # + a row for PG_NO_ROW
        self.W = torch.randn(d, self.din, generator=gen, device=device) / self.din ** 0.5
        self.refresh()

    def refresh(self):
        self.T16, self.W16 = self.T[:-1].bfloat16(), self.W.bfloat16()

    def buffers(self, N):
        dev = self.E.device
        size = pg.gather_project_workspace_size(N, self.d, 0, pg.GATE_SCALAR)
        return (torch.empty(N, self.d, dtype=torch.bfloat16, device=dev),
                torch.empty(N, self.din, dtype=torch.bfloat16, device=dev),
                torch.empty(N, self.d, dtype=torch.bfloat16, device=dev),
                torch.empty(size // 4 + 4, device=dev))

    def forward(self, tokens, bufs):
        x, e, y, ws = bufs
        pg.embed(tokens, self.E, x, self.vocab, scale=self.scale)
        pg.gather_project_gate(self.desc, tokens, self.T16, e, self.W16, self.d, pg.GATE_SCALAR, y, ws, g=self.g,
                               x_resid=x)
        return e, y


def train(steps=40, n_tokens=8192, seed=0, device="cuda"):
    """Returns the loss of every step (a device tensor)."""
    w = W.make_workload(2)
    spec = W.TableSpec("memory", W.MODE_PAGEGRAM, K=8, S=4, r=64, row_dtype=W.DT_BF16, pages=[499, 491], hash_seed=7)
    vocab, d = 512, 256
    B, L = 8, n_tokens // 8
    rng = np.random.default_rng(seed)
    tokens = torch.from_numpy(W.zipf_ids(rng, vocab, w.zipf_s, B * L).reshape(B, L)).to(device)
    N = B * L
    teacher = Memory(spec, vocab, d, seed + 1, device, std=1.0)
    student = Memory(spec, vocab, d, seed + 2, device, std=0.1)
    bufs = student.buffers(N)
    target = teacher.forward(tokens, teacher.buffers(N))[1].float()

    reads = N * len(spec.orders) * spec.K
    rows = torch.empty(reads, dtype=torch.int32, device=device)
    dT = torch.empty(reads, spec.r, device=device)
    count = torch.empty(1, dtype=torch.int32, device=device)
    dE = torch.empty_like(student.E)
    ws_rows = torch.empty(pg.lookup_grad_workspace_size(student.desc, N), dtype=torch.uint8, device=device)
    ws_emb = torch.empty(pg.embed_grad_workspace_size(N, vocab, d), dtype=torch.uint8, device=device)
    ws_orth = torch.empty(pg.orthogonalize_workspace_size(1, d, student.din), dtype=torch.uint8, device=device)
    momentum = torch.zeros_like(student.W)
    update = torch.empty(d, student.din, dtype=torch.bfloat16, device=device)
    freq = torch.bincount(tokens.view(-1).long(), minlength=vocab).clamp(min=1)[:, None]
    losses = torch.empty(steps, device=device)
    for step in range(steps):
        e, y = student.forward(tokens, bufs)
        diff = y.float() - target
        losses[step] = diff.square().mean()
        dy = diff.bfloat16()
        dW = student.g * (dy.T @ e).float()
        de = student.g * (dy @ student.W16)
        pg.embed_grad(tokens, dy, dE, vocab, ws_emb, scale=student.scale)
        pg.lookup_grad(student.desc, tokens, de, rows, dT, count, ws_rows)
        momentum.mul_(0.9).add_(dW)
        pg.orthogonalize(momentum, update, ws_orth, scale=max(1.0, d / student.din) ** 0.5)

        student.E.sub_(dE / freq, alpha=0.5 / student.scale ** 2)
        at = torch.where(rows < 0, student.T.shape[0] - 1, rows.long())  # PG_NO_ROW: the spare row
        norm = dT.square().mean(1, keepdim=True).sqrt().add_(1e-3)
        student.T.index_add_(0, at, dT / norm, alpha=-0.1)
        student.W.sub_(update.float(), alpha=0.01)
        student.refresh()
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=8192)
    a = ap.parse_args()
    losses = train(a.steps, a.tokens).tolist()
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}")
    if pg.device_error() != 0:
        raise RuntimeError("device-side wait gave up")


if __name__ == "__main__":
    main()
