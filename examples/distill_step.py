"""Distillation into a small mixture of experts, trained on compressed gradients.

One step, as data-parallel training runs it (the workers are simulated on one
GPU): the teacher answers each worker's tokens with row packets of its top
logits (``logits_topk``); the student's loss against them and the router's
balance loss come with their gradients (``distill_loss_grad``,
``balance_loss_grad``), which PyTorch carries back to the parameters; each
worker's flat gradient is compressed to a packet with its residual kept
(``topk_compress``), and the packets are summed and applied
(``sparse_aggregate_apply``).

    python examples/distill_step.py [steps]
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import error_feedback_gradient_gb300 as efg
from error_feedback_gradient_gb300 import workloads as wl

DEV = "cuda"


class Student(torch.nn.Module):
    """Router, experts (one matrix each, the best two per token) and a head."""

    def __init__(self, width: int, experts: int, vocab: int, seed: int):
        super().__init__()
        self.shapes = [(experts, width), (experts, width, width), (vocab, width)]
        self.offsets = wl.segments_from_sizes([wl.numel(s) for s in self.shapes])
        # all parameters in one flat fp32 vector, as the compressor takes them
        self.flat = torch.nn.Parameter(
            wl.normal(self.offsets[-1], 0.05, seed, DEV))

    def forward(self, x: torch.Tensor):
        router, experts, head = (
            self.flat[a:b].view(s)
            for a, b, s in zip(self.offsets, self.offsets[1:], self.shapes))
        z = x @ router.t()
        weight, ids = torch.topk(torch.softmax(z, 1), 2, dim=1)
        y = x
        for j in range(2):
            y = y + weight[:, j:j + 1] * torch.bmm(x.unsqueeze(1), experts[ids[:, j]]).squeeze(1)
        return y @ head.t(), z, ids.to(torch.int32)


def train(steps: int = 40, workers: int = 2, tokens: int = 512, width: int = 64,
          experts: int = 8, vocab: int = 1000, k: int = 32, tau: float = 2.0,
          keep: float = 0.05, eta: float = 50.0, seed: int = 0):
    """Runs ``steps`` steps; returns (distillation loss, balance loss) per step."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    model = Student(width, experts, vocab, seed + 1)
    mix = torch.randn(width, width, generator=gen, device=DEV) / width ** 0.5
    teacher = 3.0 * torch.randn(vocab, width, generator=gen, device=DEV) / width ** 0.5

    f32, i32 = torch.float32, torch.int32
    n = model.offsets[-1]
    seg_k = [max(1, int(keep * (b - a))) for a, b in zip(model.offsets, model.offsets[1:])]
    K = sum(seg_k)
    ws = torch.empty(efg.topk_workspace_size(n, model.offsets, seg_k), dtype=torch.uint8,
                     device=DEV)
    wa = torch.empty(efg.aggregate_workspace_size(workers, efg.IDX_INT32, n),
                     dtype=torch.uint8, device=DEV)
    segments = [0, tokens // 2, tokens]                 # two sequences per worker
    wb = torch.empty(efg.balance_workspace_size(tokens, experts, 2, segments),
                     dtype=torch.uint8, device=DEV)
    residual = [torch.zeros(n, device=DEV) for _ in range(workers)]
    values = [torch.empty(K, device=DEV) for _ in range(workers)]
    index = [torch.empty(K, dtype=i32, device=DEV) for _ in range(workers)]

    packet = (torch.empty(tokens, k, device=DEV), torch.empty(tokens, k, dtype=i32, device=DEV))
    counts, tail = torch.empty(tokens, dtype=i32, device=DEV), torch.empty(tokens, device=DEV)
    row_loss = torch.empty(tokens, device=DEV)
    # a mean over the step's tokens, and tau^2 so that its size does not depend on tau
    row_grad = torch.full((tokens,), tau * tau / (tokens * workers), device=DEV)
    bal_loss = torch.empty(2, device=DEV)
    bal_counts = torch.empty(2, experts, dtype=i32, device=DEV)
    bal_tokens = torch.empty(2, dtype=i32, device=DEV)
    seg_grad = torch.full((2,), 1.0 / (2 * workers), device=DEV)

    history = []
    for _ in range(steps):
        total, balance = torch.zeros((), device=DEV), torch.zeros((), device=DEV)
        for w in range(workers):
            x = torch.randn(tokens, width, generator=gen, device=DEV)
            efg.logits_topk(torch.tanh(x @ mix) @ teacher.t(), k, tau, *packet, counts, tail)

            logits, z, ids = model(x)
            g_logits = torch.empty_like(logits)
            efg.distill_loss_grad(logits.detach(), *packet, tau, row_loss, g_logits,
                                  counts=counts, tail=tail, row_grad=row_grad)
            g_z = torch.empty_like(z)
            efg.balance_loss_grad(z.detach(), ids, segments, 0.02, 0.001, bal_loss, bal_counts,
                                  bal_tokens, g_z, seg_grad=seg_grad, workspace=wb)
            model.flat.grad = None
            torch.autograd.backward([logits, z], [g_logits, g_z])
            efg.topk_compress(model.flat.grad, residual[w], model.offsets, seg_k, values[w],
                              index[w], None, ws)
            total += tau * tau * row_loss.mean() / workers
            balance += bal_loss.mean() / workers
        efg.sparse_aggregate_apply(values, index, None, [K] * workers, n, eta, None,
                                   model.flat.data, wa)
        history.append((total, balance))
    return [(float(a), float(b)) for a, b in history]


if __name__ == "__main__":
    run = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    for i, (loss, balance) in enumerate(run):
        if i % 5 == 0 or i == len(run) - 1:
            print(f"step {i:3d}  distillation {loss:.4f}  balance {balance:.5f}")
