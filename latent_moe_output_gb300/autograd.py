"""torch.autograd wrappers of the differentiable operators around the tail.

``dispatch_rows``, ``combine_rows`` and ``residual_norm`` call the same kernels as
``block`` forward and backward; gradients flow to x, rows, weights, block, residual,
the norm weights and the gate. Second derivatives are not provided.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import block as _block


def _dense(grad):
    """A gradient as the operators take it. Autograd may pass a strided one, or a contiguous
    view whose address is not a multiple of 16."""
    grad = grad.contiguous()
    return grad if grad.data_ptr() % 16 == 0 else grad.clone()


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, expert_ids, E):
        d = _block.dispatch(x, expert_ids, E)
        ctx.mark_non_differentiable(d.offsets, d.order, d.position)
        ctx.save_for_backward(d.position)
        return d.rows, d.offsets, d.order, d.position

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_rows, *_):
        (position,) = ctx.saved_tensors
        return _block.combine(_dense(grad_rows), position), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, position, weights):
        # Only the gradient of the weights reads the rows.
        wanted = weights is not None and ctx.needs_input_grad[2]
        ctx.save_for_backward(rows if wanted else None, position, weights)
        return _block.combine(rows, position, weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        rows, position, weights = ctx.saved_tensors
        grad_rows, grad_weights = _block.combine_backward(_dense(grad_out), rows, position, weights)
        return grad_rows, None, grad_weights


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, block, residual, post_weight, next_weight, gate, eps, residual_scale):
        ctx.set_materialize_grads(False)
        out, nxt = _block.residual_norm(block, residual, post_weight, next_weight, eps, gate=gate,
                                        residual_scale=residual_scale)
        ctx.save_for_backward(block, out, post_weight, next_weight, gate)
        ctx.eps, ctx.scale = eps, residual_scale
        return out, nxt

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_next):
        block, out, post_weight, next_weight, gate = ctx.saved_tensors
        if grad_out is None and grad_next is None:
            return (None,) * 7
        if next_weight is not None:  # the next norm's output may have gone unused
            grad_next = torch.zeros_like(block) if grad_next is None else _dense(grad_next)
        if grad_out is not None:
            grad_out = _dense(grad_out)
        g = _block.residual_norm_backward(grad_out, grad_next, block, out, post_weight,
                                          next_weight, ctx.eps, gate=gate,
                                          residual_scale=ctx.scale)
        grad_block, grad_residual, grad_post, grad_gate, grad_nextw = g
        return grad_block, grad_residual, grad_post, grad_nextw, grad_gate, None, None


def dispatch_rows(x, expert_ids, E: int) -> _block.Dispatched:
    """``block.dispatch`` with a gradient for x."""
    return _block.Dispatched(*_Dispatch.apply(x, expert_ids, E))


def combine_rows(rows, position, weights=None):
    """``block.combine`` with gradients for rows and weights."""
    return _Combine.apply(rows, position, weights)


def residual_norm(block, residual, post_weight, next_weight, eps: float, gate=None,
                  residual_scale: float = 1.0):
    """``block.residual_norm`` with gradients for every tensor argument."""
    return _ResidualNorm.apply(block, residual, post_weight, next_weight, gate, eps,
                               residual_scale)
