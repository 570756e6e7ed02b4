"""One distillation step of P data-parallel workers, from hidden states to
averaged gradients: the operators that produce a worker's gradients next to
the ones that average them.

The model is the end of a language model with a router: hidden states X
[tokens, hidden] of each worker go through a vocabulary layer W [vocab,
hidden], whose logits are distilled from a teacher's top logits, and through a
router R [experts, hidden], whose choices the balance loss evens out over all
workers.  Per step:

  1. once: W and R to 8 bits in both orders                     gar_fp8_quantize (square blocks)
  2. per worker: X to 8 bits in both orders; the logits          gar_fp8_quantize, gar_fp8_matmul
     z = X W^T (bf16) and r = X R^T (fp32); the distillation     gar_distill_loss
     loss, its gradient over z; that gradient to 8 bits in       gar_fp8_quantize (e5m2)
     both orders; dW = dz^T X (fp32, into the worker's flat      gar_fp8_matmul
     gradient buffer) and dX = dz W (bf16)                       gar_fp8_matmul
  3. over all workers: choices, counts, balance loss, its        gar_balance_loss
     gradient over r
  4. per worker: that gradient to 8 bits; dR = dr^T X (into      gar_fp8_quantize, gar_fp8_matmul
     the flat buffer), dX += dr R                                gar_fp8_matmul (c = d)
  5. the averaging step over the flat gradient buffers:          pipeline.AveragingStep
     exact and compressed averages, NMSE

Everything here is host-side orchestration on the caller's current stream;
each step of the arithmetic runs in the library's CUDA kernels.  Buffers are
allocated once, at construction; a step allocates nothing on the device.
"""
from __future__ import annotations

import numpy as np

from . import (fp8_matrix, gar_balance_loss, gar_balance_workspace_bytes, gar_distill_loss, gar_fp8_matmul,
               gar_fp8_quantize, pointer_table)
from .pipeline import AveragingStep, flat_offsets


class StudentStep:
    """Device-resident state of the step.

    head [vocab, hidden], router [experts, hidden]: fp32 CUDA tensors, the
    weights (read every step; whoever updates them does so between steps).
    P workers of ``tokens`` tokens each; k choices a token; alpha the balance
    loss's weight; tau the distillation's temperature.

    The objective is F = (1 / P) sum over workers of D_w + alpha B, with D_w a
    worker's distillation losses summed with its tokens' weights and B the
    balance loss over all workers' tokens.  As the averages divide by P, each
    worker's gradients are those of P F = sum of D_w + P alpha B, as far as
    its own tokens go.  After ``run(...)``:

      loss[w]            the tokens' distillation losses (without their weights)
      choice[w], counts  the router's choices
      balance            P alpha B: F is the workers' mean of D_w + balance / P
      dx[w]              the gradient of P F over the worker's hidden states
      grads[w]           the worker's share of P F's gradient over the weights, flat
                         (head_grad[w] and router_grad[w] are views of it)
      averaging          ring_flat[w] and thc_flat: the averages of grads, the
                         gradient of F, exact and compressed
    """

    def __init__(self, head, router, *, workers: int, tokens: int, k: int = 2, alpha: float = 0.01, tau: float = 1.0,
                 bits: int = 4):
        import torch

        self.torch, self.P, self.tokens, self.k, self.alpha, self.tau = torch, workers, tokens, k, float(alpha), float(tau)
        self.head, self.router = head, router
        (vocab, hidden), (experts, same) = head.shape, router.shape
        if same != hidden:
            raise ValueError(f"head and router have different hidden sizes: {hidden} and {same}")
        dev, e5m2 = head.device, torch.float8_e5m2

        def both(rows, cols, dtype=None):  # a matrix and its transpose, with their scales
            return (*fp8_matrix(rows, cols, dtype, dev), *fp8_matrix(cols, rows, dtype, dev))

        self.head8, self.router8 = both(vocab, hidden), both(experts, hidden)
        self.x8 = [both(tokens, hidden) for _ in range(workers)]
        self.dz8, self.dr8 = both(tokens, vocab, e5m2), both(tokens, experts, e5m2)
        self.z = torch.empty((tokens, vocab), dtype=torch.bfloat16, device=dev)  # one worker's logits, then their gradient
        self.r = [torch.empty((tokens, experts), device=dev) for _ in range(workers)]
        self.loss = [torch.empty(tokens, device=dev) for _ in range(workers)]
        self.lse = torch.empty(tokens, device=dev)
        self.choice = [torch.empty((tokens, k), dtype=torch.int32, device=dev) for _ in range(workers)]
        self.counts = torch.empty((workers, experts), dtype=torch.int32, device=dev)
        self.balance = torch.empty(1, device=dev)
        self.dx = [torch.empty((tokens, hidden), dtype=torch.bfloat16, device=dev) for _ in range(workers)]
        self.workspace = torch.empty(gar_balance_workspace_bytes(workers), dtype=torch.uint8, device=dev)
        sizes = np.array([vocab * hidden, experts * hidden], np.int64)
        offs = flat_offsets(sizes)
        self.grads = [torch.zeros(int(offs[-1]), device=dev) for _ in range(workers)]
        self.head_grad = [g[:vocab * hidden].view(vocab, hidden) for g in self.grads]
        self.router_grad = [g[int(offs[1]):int(offs[1]) + experts * hidden].view(experts, hidden) for g in self.grads]
        self.averaging = AveragingStep(self.grads, sizes, offs, b=bits)
        self._r_table, self._choice_table = pointer_table(self.r), pointer_table(self.choice)

    def run(self, seed: int, hidden, index, teacher, weight=None, valid=None):
        """One step.  Per worker: hidden[w] [tokens, hidden] bf16 or fp32; the
        teacher's top entries index[w] int32 and teacher[w] fp32, [tokens, n];
        weight[w] [tokens] fp32, each token's share of the loss (0: padding;
        None: 1 / tokens each); valid[w] [tokens] uint8, the tokens that the
        router counts (None: all).  seed keys the compressed average's draws."""
        if weight is None:
            if not hasattr(self, "_even"):
                self._even = self.torch.full((self.tokens,), 1.0 / self.tokens, device=self.head.device)
            weight = [self._even] * self.P
        gar_fp8_quantize(self.head, *self.head8, square=True)
        gar_fp8_quantize(self.router, *self.router8, square=True)
        head, head_s, head_t, head_ts = self.head8
        router, router_s, router_t, router_ts = self.router8
        dz, dz_s, dz_t, dz_ts = self.dz8
        for w in range(self.P):
            x, x_s, x_t, x_ts = self.x8[w]
            gar_fp8_quantize(hidden[w], x, x_s, x_t, x_ts)
            gar_fp8_matmul(x, x_s, head, head_s, self.z)
            gar_fp8_matmul(x, x_s, router, router_s, self.r[w])
            gar_distill_loss(self.z, index[w], teacher[w], self.tau, self.loss[w], self.lse, dz=self.z, weight=weight[w])
            gar_fp8_quantize(self.z, dz, dz_s, dz_t, dz_ts)
            gar_fp8_matmul(dz_t, dz_ts, x_t, x_ts, self.head_grad[w])
            gar_fp8_matmul(dz, dz_s, head_t, head_ts, self.dx[w])
        # the averages divide by P what the workers' gradients of one pooled loss would add up to
        gar_balance_loss(self._r_table, self.k, self.alpha * self.P, self._choice_table, self.counts, self.balance,
                         self.workspace, dz=self._r_table, valid=valid)
        dr, dr_s, dr_t, dr_ts = self.dr8
        for w in range(self.P):
            x, x_s, x_t, x_ts = self.x8[w]
            gar_fp8_quantize(self.r[w], dr, dr_s, dr_t, dr_ts)
            gar_fp8_matmul(dr_t, dr_ts, x_t, x_ts, self.router_grad[w])
            gar_fp8_matmul(dr, dr_s, router_t, router_ts, self.dx[w], c=self.dx[w])
        self.averaging.run(seed)
