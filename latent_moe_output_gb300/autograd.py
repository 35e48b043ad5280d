"""torch.autograd wrappers of the differentiable operators around the tail.

``dispatch_rows``, ``combine_rows``, ``residual_norm`` and ``expert_ffn`` call the same
kernels as ``block`` and ``experts`` forward and backward; gradients flow to x, rows,
weights, block, residual, the norm weights and the gate. Second derivatives are not
provided.
"""

from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import block as _block
from . import experts as _experts


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


_SAVE = ("bf16", "8bit", "all8bit")


class _ExpertFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, up, down, offsets, activation, save):
        N, F = x.shape[0], up.shape[1] // 2
        grads = save is not None and any(ctx.needs_input_grad[:3])
        kept = None
        if grads:
            kept = torch.empty(N, 2, F, dtype=torch.bfloat16, device=x.device) \
                if save == "bf16" else _experts.Checkpoint8.empty(N, 2, F, device=x.device)
        hidden = _experts.expert_gated(x, up, offsets, activation=activation, saved=kept)
        out = _experts.expert_matmul(hidden, down, offsets)
        if grads:
            rows = None  # only the gradient of up reads them
            if ctx.needs_input_grad[1]:
                rows = _experts.quantize8(x) if save == "all8bit" else x
            ctx.packed = isinstance(kept, tuple), isinstance(rows, tuple)
            ctx.save_for_backward(up, down, offsets,
                                  *(kept if ctx.packed[0] else (kept, None)),
                                  *(rows if ctx.packed[1] else (rows, None)))
            ctx.activation = activation
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        up, down, offsets, kept, kept8, rows, rows8 = ctx.saved_tensors
        if ctx.packed[0]:
            kept = _experts.Checkpoint8(kept, kept8)
        grad_out = _dense(grad_out)
        want_x, want_up, want_down = ctx.needs_input_grad[:3]
        grad_x = grad_up = grad_down = None
        if want_x or want_up:
            grad_hidden, _ = _experts.expert_matmul_backward(grad_out, None, down, offsets)
            x = None
            if want_up:
                x = _experts.dequantize8(_experts.Checkpoint8(rows, rows8)) if ctx.packed[1] \
                    else rows
            grad_x, grad_up, hidden = _experts.expert_gated_backward(
                grad_hidden, x, up if want_x else None, kept, offsets,
                activation=ctx.activation, hidden=None if want_down else False)
        else:
            _, _, hidden = _experts.expert_gated_backward(None, None, None, kept, offsets,
                                                          activation=ctx.activation)
        if want_down:
            _, grad_down = _experts.expert_matmul_backward(grad_out, hidden, None, offsets)
        return grad_x, grad_up, grad_down, None, None, None


def expert_ffn(x, up, down, offsets=None, activation: str = "silu", save: str = "bf16"):
    """A gated feed-forward block for rows sorted by expert (or, without ``offsets``, one
    dense block): ``expert_matmul(expert_gated(x, up), down)`` with gradients for x [N, C],
    up [E, 2F, C] and down [E, M, F].

    ``save`` says what the backward pass reads: "bf16" keeps x and both projections in
    bf16, "8bit" the projections in 8 bits, "all8bit" x too (per row 2C + 4F, 2C + 2.13F
    and 1.06C + 2.13F bytes). The product of the block is computed again from them for the
    gradient of down: from 8 bits it is not quite the product that went forward. Error of the
    gradients of x, up and down for normal values, as a share of their norms: 0.34, 0.34 and
    0.35 % with "bf16", 0.9, 0.9 and 1.1 % with "8bit", 0.9, 1.2 and 1.1 % with "all8bit".
    Nothing is kept where gradients are off (``torch.no_grad``, ``torch.inference_mode``)."""
    if save not in _SAVE:
        raise ValueError(f"save: expected one of {_SAVE}, got {save!r}")
    # (within the function gradients are always off, and needs_input_grad goes by the tensors)
    return _ExpertFFN.apply(x, up, down, offsets, activation,
                            save if torch.is_grad_enabled() else None)


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
