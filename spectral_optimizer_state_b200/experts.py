"""Products with a mixture of experts' stacked weights, differentiable.

The weights a mixture-of-experts layer stacks are per-expert projections, which Muon steps one
matrix at a time (``MuonAdamW(..., stacked=True)``); this is the layer's side of them.  Both
directions and the weight gradient run in libmuon's kernels (include/muon.h, muon_expert_matmul and
muon_expert_grad); nothing is computed here.
"""
from __future__ import annotations

import functools


@functools.lru_cache(maxsize=1)
def _function():
    """The autograd function (torch is imported on first use, as everywhere in this package)."""
    import torch

    class _ExpertLinear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, offsets, muon, grad_into):
            ctx.save_for_backward(x, w, offsets)
            ctx.muon, ctx.grad_into = muon, grad_into
            return muon.expert_matmul(x, w, offsets)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dy):
            x, w, offsets = ctx.saved_tensors
            dx = dw = None
            if ctx.needs_input_grad[0]:
                dx = ctx.muon.expert_matmul(dy, w, offsets, transpose=True)
            if ctx.needs_input_grad[1]:
                if ctx.grad_into is not None:
                    ctx.muon.expert_grad(dy, x, offsets, ctx.grad_into, beta=1.0)
                else:
                    dw = ctx.muon.expert_grad(dy, x, offsets)
            return dx, dw, None, None, None

    return _ExpertLinear


def expert_linear(x, w, offsets, muon, grad_into=None):
    """y[t] = w[e] @ x[t] for the rows t of expert e, with gradients for x and w.

    x: [tokens, cols], rows sorted by expert; w: [experts, rows, cols]; offsets: int32 CUDA
    [experts + 1] (rows offsets[e] .. offsets[e+1]-1 belong to expert e; rows of no expert give and
    receive zeros, and so does everything if the offsets are bad, which muon.status() reports); muon:
    the libmuon context whose scratch the products use.  bf16 or fp32.
    fp32 operands, and bf16 ones whose rows do not start on 16-byte boundaries, may be repacked into that scratch
    (up to 6 bytes an element of x and w, held until the context is closed), so layers that run at the same time on
    different streams, backward passes and replayed graphs included, need a context each.
    grad_into: an fp32 [experts, rows, cols] buffer that the weight gradient is added to, over as many
    backward passes as one likes, if w requires a gradient.  w.grad then stays None, so an optimizer that
    reads it passes w over: hand the buffer to ``MuonAdamW.step`` as w's gradient, or name it in
    ``torch_optimizer(..., main_grads={name: buffer})``.
    """
    return _function().apply(x, w, offsets, muon, grad_into)
