"""torch.autograd wrapper: mean cross-entropy of E C^T over non-ignored tokens.

The forward keeps only the per-token log-sum-exp and largest logit (2N
floats) for the backward pass, which recomputes the logit tiles on chip; the
N x V logits are never stored.  The largest logits let the gradient filter's
pre-pass prove more token blocks negligible.  The mean reduction and the dtype cast of the gradients are the
caller-side plumbing around the two C-ABI calls.
"""
from __future__ import annotations

import torch

from . import backward as _cce_backward
from . import forward as _cce_forward
from ._distill import distill_backward as _distill_backward
from ._distill import distill_forward as _distill_forward


class LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, E, C, y, ignore_index: int, filter_eps: float):
        row_max = torch.empty(E.shape[0], dtype=torch.float32, device=E.device)
        loss, lse = _cce_forward(E.contiguous(), C.contiguous(), y.contiguous(), ignore_index, row_max=row_max)
        keep = y != ignore_index
        n = keep.sum()
        ctx.save_for_backward(E, C, y, lse, row_max, keep, n)
        ctx.ignore_index = ignore_index
        ctx.filter_eps = filter_eps
        return loss.sum() / n

    @staticmethod
    def backward(ctx, g):
        E, C, y, lse, row_max, keep, n = ctx.saved_tensors
        dloss = keep.to(torch.float32) * (g.to(torch.float32) / n.to(torch.float32))
        dE, dC = _cce_backward(E.contiguous(), C.contiguous(), y.contiguous(), lse, dloss.contiguous(),
                               ctx.filter_eps, ctx.ignore_index, row_max=row_max)
        return dE.to(E.dtype), dC.to(C.dtype), None, None, None


class LinearDistillation(torch.autograd.Function):
    """Mean distillation loss over the tokens with a teacher entry; the
    forward keeps the log-sum-exp (N floats) for the backward pass, which sums
    in a fixed order: the same inputs give the same gradients."""

    @staticmethod
    def forward(ctx, E, C, ids, teacher, temperature: float, ignore_index: int):
        E, C, ids, teacher = E.contiguous(), C.contiguous(), ids.contiguous(), teacher.contiguous()
        mean, inv_count = (torch.empty((), dtype=torch.float32, device=E.device) for _ in range(2))
        _, lse = _distill_forward(E, C, ids, teacher, temperature, ignore_index, mean=(mean, inv_count))
        ctx.save_for_backward(E, C, ids, teacher, lse, inv_count)
        ctx.temperature = temperature
        ctx.ignore_index = ignore_index
        return mean

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, g):
        E, C, ids, teacher, lse, inv_count = ctx.saved_tensors
        dE, dC = _distill_backward(E, C, ids, teacher, lse, g.to(torch.float32), ctx.temperature, ctx.ignore_index,
                                   bf16_grads=True, deterministic=True, dloss_scale=inv_count)
        need = ctx.needs_input_grad
        return dE if need[0] else None, dC if need[1] else None, None, None, None, None
