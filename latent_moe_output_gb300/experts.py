"""ctypes binding of the bf16 experts and of activations in 8 bits
(``include/latent_tail.h``), as ``block`` for the other operators around the tail.

    dispatch -> expert_gated -> expert_matmul -> combine
             <- expert_gated_backward <- expert_matmul_backward <-

Argument marshalling only: shapes are read from the tensors; outputs can be passed in
and are allocated with torch when they are not; a non-OK status raises
``LatentTailError``. Calls are asynchronous on ``stream`` (default: torch's current
stream); tensors allocated here belong to that stream.
"""

from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from .binding import load_library
from .block import (_BF16, _I32, _INT_MAX, _U8, _call, _empty, _index, _ptr, _shape, _size,
                    _workspace)

_I8 = torch.int8
_ACTIVATIONS = {"silu": 0, "gelu": 1}
_SAVED_NONE, _SAVED_BF16, _SAVED_8BIT = range(3)
GROUP8 = 16  # columns that share an exponent


class Checkpoint8(NamedTuple):
    """Activations in 8 bits: ``values * 2 ** (exponents - 127)``, one exponent per 16
    columns of the last dimension. Exponent 0 is a group of zeros, 255 one that held an
    infinity or a NaN (read back as NaNs). bf16's two largest magnitudes read back as
    infinities in a group that holds the largest. See latent_tail_quantize8."""

    values: torch.Tensor     # [..., C] int8
    exponents: torch.Tensor  # [..., ceil(C / 16)] uint8

    @classmethod
    def empty(cls, *shape, device="cuda"):
        """Buffers for activations of ``shape``."""
        return cls(torch.empty(*shape, dtype=_I8, device=device),
                   torch.empty(*shape[:-1], -(-shape[-1] // GROUP8), dtype=_U8, device=device))


def _activation(name) -> int:
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation: expected one of {sorted(_ACTIVATIONS)}, got {name!r}") \
            from None


def _unwanted(grad, name, operand, operand_name):
    if grad is not None and operand is None:
        raise ValueError(f"{name} given without {operand_name}")


def _saved(saved, N, F, i):
    """Kind and addresses of kept projections."""
    if saved is None:
        return _SAVED_NONE, 0, 0
    if isinstance(saved, tuple):
        if len(saved) != 2:
            raise TypeError("saved: expected Checkpoint8 or a torch.Tensor")
        return (_SAVED_8BIT, _ptr(saved[0], "saved.values", _I8, (N, 2, F), i),
                _ptr(saved[1], "saved.exponents", _U8, (N, 2, -(-F // GROUP8)), i))
    return _SAVED_BF16, _ptr(saved, "saved", _BF16, (N, 2, F), i), 0


def expert_gated(x, weights, offsets=None, activation="silu", hidden=None, saved=None,
                 stream=None):
    """hidden[r] = a(g) * u with g = weights[e, :F] @ x[r] and u = weights[e, F:] @ x[r] for
    the rows r of expert e (``offsets`` of ``dispatch``, or of some of its experts: a slice
    that begins at a multiple of four experts, or a copy of another, for the alignment to 16
    bytes; None with one matrix: every row); zeros for rows that no expert owns.

    x [N, C] bf16, weights [E, 2F, C] bf16, activation "silu" or "gelu" (its tanh form).
    ``saved`` takes g and u for the backward pass: a bf16 tensor [N, 2, F], or
    ``Checkpoint8.empty(N, 2, F)`` for 8 bits. Returns hidden [N, F]. See
    latent_tail_expert_gated."""
    N, C = _shape(x, "x", 2)
    i = _index(x, "x")
    E, F2, _ = _shape(weights, "weights", 3)
    if F2 % 2:
        raise ValueError(f"weights: expected gate and up rows, got {F2}")
    F, act = F2 // 2, _activation(activation)
    kind, values, exponents = _saved(saved, N, F, i)
    if hidden is None:
        hidden = _empty((N, F), _BF16, i, stream)
    _call("latent_tail_expert_gated", i, stream, _ptr(x, "x", _BF16, (N, C), i),
          _ptr(weights, "weights", _BF16, (E, F2, C), i),
          _ptr(offsets, "offsets", _I32, (E + 1,), i), _ptr(hidden, "hidden", _BF16, (N, F), i),
          values, exponents, N, E, F, C, act, kind)
    return hidden


@functools.lru_cache(maxsize=256)
def expert_gated_backward_workspace_size(N: int, F: int) -> int:
    return int(load_library().latent_tail_expert_gated_backward_workspace_size(N, F))


def expert_gated_backward(grad_hidden, x, weights, saved, offsets=None, activation="silu",
                          grad_x=None, grad_weights=None, hidden=None, workspace=None,
                          stream=None):
    """(grad_x, grad_weights, hidden) of ``expert_gated`` from the projections it kept in
    ``saved``; hidden is the product computed again from them (for the gradient of the
    product behind it), None where ``hidden`` is False.

    Without ``weights`` (None) grad_x is None, without ``x`` grad_weights is; without
    ``grad_hidden`` only hidden is computed. grad_weights has zeros for experts without
    rows, grad_x and hidden for rows that no expert owns. See
    latent_tail_expert_gated_backward."""
    act = _activation(activation)
    kept = saved[0] if isinstance(saved, tuple) and saved else saved
    N, two, F = _shape(kept, "saved", 3)
    if two != 2:
        raise ValueError(f"saved: expected shape (N, 2, F), got {tuple(kept.shape)}")
    i = _index(kept, "saved")
    E, C = 1, 8  # of a call that computes hidden alone
    if grad_hidden is None:
        x = weights = None
    if weights is not None:
        E, _, C = _shape(weights, "weights", 3)
    elif x is not None:
        C = _shape(x, "x", 2)[1]
    if offsets is not None:
        E = _shape(offsets, "offsets", 1)[0] - 1
    kind, values, exponents = _saved(saved, N, F, i)
    given = (_ptr(grad_hidden, "grad_hidden", _BF16, (N, F), i), _ptr(x, "x", _BF16, (N, C), i),
             _ptr(weights, "weights", _BF16, (E, 2 * F, C), i), values, exponents,
             _ptr(offsets, "offsets", _I32, (E + 1,), i))
    _unwanted(grad_x, "grad_x", weights, "weights")
    _unwanted(grad_weights, "grad_weights", x, "x")
    if weights is not None and grad_x is None:
        grad_x = _empty((N, C), _BF16, i, stream)
    if x is not None and grad_weights is None:
        grad_weights = _empty((E, 2 * F, C), _BF16, i, stream)
    if hidden is False:
        hidden = None
    elif hidden is None:
        hidden = _empty((N, F), _BF16, i, stream)
    ws = ws_bytes = 0
    if weights is not None or x is not None:
        if workspace is None:
            need = max(256, expert_gated_backward_workspace_size(N, F))
            workspace = _empty((need,), _U8, i, stream)
        ws, ws_bytes = _workspace(workspace, i)
    _call("latent_tail_expert_gated_backward", i, stream, *given,
          _ptr(grad_x, "grad_x", _BF16, (N, C), i),
          _ptr(grad_weights, "grad_weights", _BF16, (E, 2 * F, C), i),
          _ptr(hidden, "hidden", _BF16, (N, F), i), N, E, F, C, act, kind, ws, ws_bytes)
    return grad_x, grad_weights, hidden


def expert_matmul(x, weights, offsets=None, out=None, stream=None):
    """out[r] = weights[e] @ x[r] for the rows r of expert e (``offsets`` as for
    ``expert_gated``); zeros for rows that no expert owns. x [N, C], weights [E, M, C],
    out [N, M], all bf16. See latent_tail_expert_matmul."""
    N, C = _shape(x, "x", 2)
    i = _index(x, "x")
    E, M, _ = _shape(weights, "weights", 3)
    if out is None:
        out = _empty((N, M), _BF16, i, stream)
    _call("latent_tail_expert_matmul", i, stream, _ptr(x, "x", _BF16, (N, C), i),
          _ptr(weights, "weights", _BF16, (E, M, C), i),
          _ptr(offsets, "offsets", _I32, (E + 1,), i), _ptr(out, "out", _BF16, (N, M), i),
          N, E, M, C)
    return out


def expert_matmul_backward(grad_out, x, weights, offsets=None, grad_x=None, grad_weights=None,
                           stream=None):
    """(grad_x, grad_weights) of ``expert_matmul``. Without ``weights`` (None) grad_x is
    None, without ``x`` grad_weights is (not both). See latent_tail_expert_matmul_backward."""
    N, M = _shape(grad_out, "grad_out", 2)
    i = _index(grad_out, "grad_out")
    if x is None and weights is None:
        raise ValueError("x and weights are both None: no gradient to compute")
    E = 1
    if weights is not None:
        E, _, C = _shape(weights, "weights", 3)
    else:
        C = _shape(x, "x", 2)[1]
    if offsets is not None:
        E = _shape(offsets, "offsets", 1)[0] - 1
    given = (_ptr(grad_out, "grad_out", _BF16, (N, M), i), _ptr(x, "x", _BF16, (N, C), i),
             _ptr(weights, "weights", _BF16, (E, M, C), i),
             _ptr(offsets, "offsets", _I32, (E + 1,), i))
    _unwanted(grad_x, "grad_x", weights, "weights")
    _unwanted(grad_weights, "grad_weights", x, "x")
    if weights is not None and grad_x is None:
        grad_x = _empty((N, C), _BF16, i, stream)
    if x is not None and grad_weights is None:
        grad_weights = _empty((E, M, C), _BF16, i, stream)
    _call("latent_tail_expert_matmul_backward", i, stream, *given,
          _ptr(grad_x, "grad_x", _BF16, (N, C), i),
          _ptr(grad_weights, "grad_weights", _BF16, (E, M, C), i), N, E, M, C)
    return grad_x, grad_weights


def _rows(t, name):
    """Rows and columns of a tensor of at least two dimensions, its shape, and that of its
    exponents."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) == 2:
        rows, C = shape
    elif len(shape) > 2:
        rows, C = 1, shape[-1]
        for n in shape[:-1]:
            rows *= n
    else:
        raise ValueError(f"{name}: expected at least 2 dimensions, got {len(shape)}")
    if rows > _INT_MAX or C > _INT_MAX:
        _size(max(rows, C), name)
    return rows, C, shape, (*shape[:-1], -(-C // GROUP8))


def quantize8(x, out=None, stream=None) -> Checkpoint8:
    """``x`` [..., C] bf16 in 8 bits (``out``: buffers of an earlier call, or of
    ``Checkpoint8.empty``). See latent_tail_quantize8."""
    T, C, shape, eshape = _rows(x, "x")
    i = _index(x, "x")
    if out is None:
        out = Checkpoint8(_empty(shape, _I8, i, stream), _empty(eshape, _U8, i, stream))
    values, exponents = out
    _call("latent_tail_quantize8", i, stream, _ptr(x, "x", _BF16, shape, i),
          _ptr(values, "out.values", _I8, shape, i),
          _ptr(exponents, "out.exponents", _U8, eshape, i), T, C)
    return out if isinstance(out, Checkpoint8) else Checkpoint8(values, exponents)


def dequantize8(checkpoint, out=None, stream=None):
    """The activations that ``checkpoint`` stands for, [..., C] bf16 (exact: an integer of
    8 bits times a power of two). See latent_tail_dequantize8."""
    values, exponents = checkpoint
    T, C, shape, eshape = _rows(values, "checkpoint.values")
    i = _index(values, "checkpoint.values")
    if out is None:
        out = _empty(shape, _BF16, i, stream)
    _call("latent_tail_dequantize8", i, stream, _ptr(values, "checkpoint.values", _I8, shape, i),
          _ptr(exponents, "checkpoint.exponents", _U8, eshape, i),
          _ptr(out, "out", _BF16, shape, i), T, C)
    return out
