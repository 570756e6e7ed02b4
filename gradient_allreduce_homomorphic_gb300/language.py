"""One language-model training step of P data-parallel workers, from hidden
states to averaged and clipped gradients: a router with its experts and a
vocabulary layer, the operators that produce their gradients, and the ones that
average and clip them.

The model is the end of a language model: hidden states X [tokens, hidden] of
each worker pass a mixture of experts, h = X + sum over a token's choices of
weight * (x U_e^T), and then a vocabulary layer W [vocab, hidden] whose logits
are held against the next tokens.  The choices come from a router R [experts,
hidden], the weights are the softmax over a token's chosen router logits, and a
balance loss over all workers' tokens evens the choices out.  An expert takes
``capacity`` tokens of a worker at most; what is over them passes by X alone.
Per step:

  1. once: R and the experts to 8 bits in both orders           gar_fp8_quantize (square blocks)
  2. per worker: X to 8 bits in both orders; router logits       gar_fp8_quantize, gar_fp8_matmul
     r = X R^T (fp32)
  3. over all workers: choices, counts, balance loss and its     gar_balance_loss
     gradient over r; the choices' weights                       gar_expert_weights
  4. per worker: its tokens sorted by expert, their rows;        gar_expert_sort, gar_expert_gather
     per expert its rows' product; the rows back to the tokens   gar_fp8_quantize, gar_fp8_matmul
     with weights and X added (h, bf16)                          gar_expert_combine
  5. per worker: the vocabulary layer's loss, its gradient       gar_vocab_loss, gar_vocab_grad_with_loss
     over h (dX so far) and over W (fp32, into the worker's
     flat gradient buffer)
  6. per worker: the gradient over the rows and the weights;     gar_expert_combine_grad
     per expert dU (into the flat buffer) and its rows'          gar_fp8_quantize, gar_fp8_matmul
     gradient; these back to the tokens, added to dX             gar_expert_combine
  7. over all workers: the weights' gradient added to that of    gar_expert_weights_grad
     the balance loss over r
  8. per worker: dR = dr^T X (into the flat buffer), dX += dr R  gar_fp8_quantize, gar_fp8_matmul
  9. the averaging step over the flat gradient buffers, the      pipeline.AveragingStep
     averages clipped by their norm                              (gar_grad_clip)

Everything here is host-side orchestration on the caller's current stream;
each step of the arithmetic runs in the library's CUDA kernels.  Buffers are
allocated once, at construction; a step allocates nothing on the device.
"""
from __future__ import annotations

import numpy as np

from . import (fp8_matrix, gar_balance_loss, gar_balance_workspace_bytes, gar_expert_combine, gar_expert_combine_grad,
               gar_expert_gather, gar_expert_rows, gar_expert_sort, gar_expert_weights, gar_expert_weights_grad,
               gar_expert_workspace_bytes, gar_fp8_matmul, gar_fp8_quantize, gar_vocab_grad_with_loss,
               gar_vocab_loss, gar_vocab_workspace_bytes, pointer_table)
from .pipeline import AveragingStep, flat_offsets


class LanguageStep:
    """Device-resident state of the step.

    head [vocab, hidden] bf16, router [experts, hidden] and experts [experts,
    hidden, hidden] fp32 CUDA tensors, the weights (read every step; whoever
    updates them does so between steps).  hidden has to be a multiple of 8.  P
    workers of ``tokens`` tokens each; k choices a token; capacity: rows of an
    expert for one worker's tokens; alpha the balance loss's weight; max_norm:
    what the averaged gradients' norm is clipped to (None: not at all).

    The objective is F = (1 / P) sum over workers of L_w + alpha B, with L_w a
    worker's cross entropies summed with its tokens' weights and B the balance
    loss over all workers' tokens.  As the averages divide by P, each worker's
    gradients are those of P F, as far as its own tokens go.  After ``run(...)``:

      loss[w]               the tokens' cross entropies (0 where a token does not count)
      choice[w], position[w], counts   the router's choices, their rows (-1: none)
      balance               P alpha B
      dx[w]                 the gradient of P F over the worker's hidden states
      grads[w]              the worker's share of P F's gradient over the weights, flat
                            (head_grad[w], router_grad[w], expert_grad[w] are views of it)
      averaging             ring_flat[w] and thc_flat: the averages of grads, exact and
                            compressed, clipped; averaging.norm: the exact one's norm
    """

    def __init__(self, head, router, experts, *, workers: int, tokens: int, k: int = 2, capacity: int = 0, alpha: float = 0.01,
                 bits: int = 4, max_norm=None):
        import torch

        self.torch, self.P, self.tokens, self.k, self.alpha = torch, workers, tokens, k, float(alpha)
        self.head, self.router, self.experts = head, router, experts
        (vocab, hidden), (E, same), shape = head.shape, router.shape, tuple(experts.shape)
        if same != hidden or shape != (E, hidden, hidden) or hidden % 8:
            raise ValueError(f"head {tuple(head.shape)}, router {tuple(router.shape)} and experts {shape} do not fit together, "
                             "or their hidden size is not a multiple of 8")
        self.E, self.capacity = E, int(capacity) or 2 * -(-tokens * k // E)
        dev, bf16, e5m2 = head.device, torch.bfloat16, torch.float8_e5m2
        C, rows = self.capacity, gar_expert_rows(1, tokens, k, E, capacity=self.capacity)

        def both(n, m, dtype=None):  # a matrix and its transpose, with their scales
            return (*fp8_matrix(n, m, dtype, dev), *fp8_matrix(m, n, dtype, dev))

        def each(*shape, dtype=torch.float32):
            return [torch.empty(shape, dtype=dtype, device=dev) for _ in range(workers)]

        self.router8, self.expert8 = both(E, hidden), [both(hidden, hidden) for _ in range(E)]
        self.x8, self.dr8 = [both(tokens, hidden) for _ in range(workers)], both(tokens, E, e5m2)
        self.rows8, self.drows8 = [both(C, hidden) for _ in range(E)], both(C, hidden, e5m2)
        self.r, self.dr = each(tokens, E), each(tokens, E)
        self.choice, self.position = each(tokens, k, dtype=torch.int32), each(tokens, k, dtype=torch.int32)
        self.weight, self.dweight = each(tokens, k), each(tokens, k)
        self.counts = torch.empty((workers, E), dtype=torch.int32, device=dev)
        self.balance = torch.empty(1, device=dev)
        self.source = torch.empty(rows, dtype=torch.int32, device=dev)  # one worker's, as the rows below
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        self.xs, self.ys = (torch.empty((rows, hidden), dtype=bf16, device=dev) for _ in range(2))
        self.h, self.dx = each(tokens, hidden, dtype=bf16), each(tokens, hidden, dtype=bf16)
        self.loss, self.lse = each(tokens), each(tokens)
        self._even = torch.full((tokens,), 1.0 / max(tokens, 1), device=dev)  # the weights where none are given
        self.workspace = torch.empty(max(gar_balance_workspace_bytes(workers), gar_expert_workspace_bytes(1, tokens, k, E),
                                         gar_vocab_workspace_bytes(tokens, vocab, hidden, torch.float32)), dtype=torch.uint8,
                                     device=dev)
        sizes = np.array([vocab * hidden, E * hidden, E * hidden * hidden], np.int64)
        offs = flat_offsets(sizes)
        self.grads = [torch.zeros(int(offs[-1]), device=dev) for _ in range(workers)]
        view = lambda g, i, *shape: g[int(offs[i]):int(offs[i] + sizes[i])].view(*shape)  # noqa: E731
        self.head_grad = [view(g, 0, vocab, hidden) for g in self.grads]
        self.router_grad = [view(g, 1, E, hidden) for g in self.grads]
        self.expert_grad = [view(g, 2, E, hidden, hidden) for g in self.grads]
        self.averaging = AveragingStep(self.grads, sizes, offs, b=bits, max_norm=max_norm)
        self._tables = {n: pointer_table(getattr(self, n)) for n in ("r", "dr", "choice", "weight", "dweight")}

    def run(self, seed: int, hidden, target, weight=None, valid=None):
        """One step.  Per worker: hidden[w] [tokens, hidden] bf16; target[w]
        [tokens] int32, the next tokens (outside the vocabulary: does not count);
        weight[w] [tokens] fp32, each token's share of the loss (0: padding; None:
        1 / tokens each); valid[w] [tokens] uint8, the tokens that the router
        counts (None: all).  The hidden states of tokens that do not count have to
        be finite: the 8-bit products meet them with zeros.  seed keys the
        compressed average's draws."""
        if weight is None:
            weight = [self._even] * self.P
        t, C = self._tables, self.capacity
        gar_fp8_quantize(self.router, *self.router8, square=True)
        for e in range(self.E):
            gar_fp8_quantize(self.experts[e], *self.expert8[e], square=True)
        router, router_s, router_t, router_ts = self.router8
        for w in range(self.P):
            gar_fp8_quantize(hidden[w], *self.x8[w])
            gar_fp8_matmul(*self.x8[w][:2], router, router_s, self.r[w])
        # the averages divide by P what the workers' gradients of one pooled loss would add up to
        gar_balance_loss(t["r"], self.k, self.alpha * self.P, t["choice"], self.counts, self.balance, self.workspace, dz=t["dr"],
                         valid=valid)
        gar_expert_weights(t["r"], t["choice"], t["weight"])
        rows = [slice(e * C, (e + 1) * C) for e in range(self.E)]
        drows, drows_s, drows_t, drows_ts = self.drows8
        for w in range(self.P):
            choice, position, share, dshare = [self.choice[w]], [self.position[w]], [self.weight[w]], [self.dweight[w]]
            gar_expert_sort(choice, self.E, position, self.source, self.offsets, self.workspace, capacity=C)
            gar_expert_gather([hidden[w]], position, self.source, self.xs)
            for e, at in enumerate(rows):
                gar_fp8_quantize(self.xs[at], *self.rows8[e])
                gar_fp8_matmul(*self.rows8[e][:2], *self.expert8[e][:2], self.ys[at])
            gar_expert_combine(self.ys, position, [self.h[w]], weight=share, addend=[hidden[w]])
            gar_vocab_loss(self.h[w], self.head, target[w], self.loss[w], self.lse[w], self.workspace, weight=weight[w])
            gar_vocab_grad_with_loss(self.h[w], self.head, target[w], self.loss[w], self.lse[w], self.dx[w], self.head_grad[w],
                                     self.workspace, weight=weight[w])
            gar_expert_combine_grad([self.dx[w]], self.ys, position, self.source, share, self.ys, dshare)  # over the rows
            for e, at in enumerate(rows):
                gar_fp8_quantize(self.ys[at], drows, drows_s, drows_t, drows_ts)
                gar_fp8_matmul(drows_t, drows_ts, *self.rows8[e][2:], self.expert_grad[w][e])
                gar_fp8_matmul(drows, drows_s, *self.expert8[e][2:], self.xs[at])
            gar_expert_combine(self.xs, position, [self.dx[w]], addend=[self.dx[w]])
        gar_expert_weights_grad(t["weight"], t["dweight"], t["choice"], t["dr"], accumulate=True)
        dr, dr_s, dr_t, dr_ts = self.dr8
        for w in range(self.P):
            gar_fp8_quantize(self.dr[w], dr, dr_s, dr_t, dr_ts)
            gar_fp8_matmul(dr_t, dr_ts, *self.x8[w][2:], self.router_grad[w])
            gar_fp8_matmul(dr, dr_s, router_t, router_ts, self.dx[w], c=self.dx[w])
        self.averaging.run(seed)
