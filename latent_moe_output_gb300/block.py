"""ctypes binding of the operators around the tail (``include/latent_tail.h``).

    tokens -> dispatch -> experts (expert_matvec4) -> combine -> routed partial
           -> forward (the tail) -> residual_norm -> the next block

Argument marshalling only, as in ``binding``: shapes are read from the tensors;
outputs can be passed in (a decode loop keeps its buffers) and are allocated with
torch when they are not, but for ``residual_norm_backward``, which allocates its
gradients always; a non-OK status raises ``LatentTailError``. Calls are
asynchronous on ``stream`` (default: torch's current stream). Tensors allocated
here belong to that stream; a tensor of another stream must be kept alive and
ordered by the caller, as for any torch operation.
"""

from __future__ import annotations

import functools
from typing import NamedTuple, Optional

import torch

from .binding import LatentTailError, _stream_handle, load_library

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_GATE_NONE, _GATE_TOKEN, _GATE_CHANNEL, _GATE_FULL = range(4)


class Dispatched(NamedTuple):
    """Result of ``dispatch``."""

    rows: Optional[torch.Tensor]  # [T*K, L] bf16, sorted by expert; None for the sort alone
    offsets: torch.Tensor         # [E+1] int32: rows of expert e are offsets[e]:offsets[e+1]
    order: torch.Tensor           # [T*K] int32: flat choice index of each row
    position: torch.Tensor        # [T, K] int32: row of each choice, -1 - row without an expert


# A call on small tensors takes a few microseconds on the GPU, so its checks read
# each property once and the stream comes as a plain handle, without a Stream object.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_entry_points = {}


def _ptr(t, name, dtype, shape, index):
    """Device address of ``t`` after checking it; 0 for None."""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index \
                and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on CUDA device {index}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


_INT_MAX = 2 ** 31 - 1  # ctypes cuts larger sizes off without a word


def _size(n, name) -> int:
    if n > _INT_MAX:
        raise ValueError(f"{name}: sizes are at most {_INT_MAX}, got {n}")
    return n


def _shape(t, name, ndim):
    """Shape of a tensor that fixes a call's sizes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if len(shape) != ndim:
        raise ValueError(f"{name}: expected {ndim} dimensions, got {len(shape)}")
    for n in shape:
        if n > _INT_MAX:
            _size(n, name)
    return shape


def _index(t, name) -> int:
    """CUDA device index of the tensor that fixes a call's device."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return index


def _empty(shape, dtype, index, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=index)


def _like(t, stream):
    """An empty tensor like the contiguous ``t`` (half the host time of torch.empty)."""
    if stream is None:
        return torch.empty_like(t)
    return _empty(t.shape, t.dtype, t.get_device(), stream)


def _call(name, index, stream, *args):
    """Run one C entry point with ``index`` as the current device."""
    if torch._C._cuda_getDevice() != index:
        with torch.cuda.device(index):
            return _call(name, index, stream, *args)
    fn = _entry_points.get(name)
    if fn is None:
        fn = _entry_points[name] = getattr(load_library(), name)
    status = fn(*args, _raw_stream(index) if stream is None else _stream_handle(stream))
    if status:
        raise LatentTailError(status, name)


@functools.lru_cache(maxsize=256)
def dispatch_workspace_size(T: int, K: int, E: int) -> int:
    return int(load_library().latent_tail_dispatch_workspace_size(T, K, E))


def dispatch(x, expert_ids, E: int, rows=None, offsets=None, order=None, position=None,
             workspace=None, stream=None) -> Dispatched:
    """Sort the choices ``expert_ids`` [T, K] (int32; anything outside [0, E) is a
    choice without an expert) by expert and copy the rows of ``x`` [T, L] to their
    places. ``x`` None sorts alone. See latent_tail_dispatch."""
    T, K = _shape(expert_ids, "expert_ids", 2)
    _size(E, "E")
    i = _index(expert_ids, "expert_ids")
    L = 0
    if x is not None:
        L = _shape(x, "x", 2)[1]
        if rows is None:
            rows = _empty((T * K, L), _BF16, i, stream)
    elif rows is not None:
        raise ValueError("rows given without x")
    if offsets is None:
        offsets = _empty((E + 1,), _I32, i, stream)
    if order is None:
        order = _empty((T * K,), _I32, i, stream)
    if position is None:
        position = _empty((T, K), _I32, i, stream)
    ws = ws_bytes = 0
    need = dispatch_workspace_size(T, K, E)
    if need:
        if workspace is None:
            workspace = _empty((need,), _U8, i, stream)
        ws, ws_bytes = _workspace(workspace, i)
    _call("latent_tail_dispatch", i, stream,
          _ptr(x, "x", _BF16, (T, L), i), _ptr(expert_ids, "expert_ids", _I32, (T, K), i),
          _ptr(rows, "rows", _BF16, (T * K, L), i), _ptr(offsets, "offsets", _I32, (E + 1,), i),
          _ptr(order, "order", _I32, (T * K,), i), _ptr(position, "position", _I32, (T, K), i),
          T, K, E, L, ws, ws_bytes)
    return Dispatched(rows, offsets, order, position)


def _workspace(workspace, index):
    nbytes = workspace.numel() * workspace.element_size()
    return _ptr(workspace, "workspace", workspace.dtype, workspace.shape, index), nbytes


def combine(rows, position, weights=None, out=None, stream=None):
    """out[t] = sum over the routed choices k of weights[t, k] * rows[position[t, k]]
    (weights None: 1, the gradient of ``dispatch``'s copy). See latent_tail_combine."""
    T, K = _shape(position, "position", 2)
    i = _index(position, "position")
    L = _shape(rows, "rows", 2)[1]
    if out is None:
        out = _empty((T, L), _BF16, i, stream)
    _call("latent_tail_combine", i, stream, _ptr(rows, "rows", _BF16, (T * K, L), i),
          _ptr(position, "position", _I32, (T, K), i),
          _ptr(weights, "weights", _F32, (T, K), i), _ptr(out, "out", _BF16, (T, L), i), T, K, L)
    return out


def combine_backward(grad_out, rows, position, weights=None, grad_rows=None, grad_weights=None,
                     stream=None):
    """(grad_rows, grad_weights) of ``combine``. ``rows`` None: only grad_rows, with
    None for grad_weights. See latent_tail_combine_backward."""
    T, K = _shape(position, "position", 2)
    i = _index(position, "position")
    L = _shape(grad_out, "grad_out", 2)[1]
    if grad_rows is None:
        grad_rows = _empty((T * K, L), _BF16, i, stream)
    if grad_weights is None and rows is not None:
        grad_weights = _empty((T, K), _F32, i, stream)
    _call("latent_tail_combine_backward", i, stream,
          _ptr(grad_out, "grad_out", _BF16, (T, L), i), _ptr(rows, "rows", _BF16, (T * K, L), i),
          _ptr(position, "position", _I32, (T, K), i), _ptr(weights, "weights", _F32, (T, K), i),
          _ptr(grad_rows, "grad_rows", _BF16, (T * K, L), i),
          _ptr(grad_weights, "grad_weights", _F32, (T, K), i), T, K, L)
    return grad_rows, grad_weights


def expert_matvec4(x, packed, scales, offsets=None, out=None, stream=None):
    """out[r, m] = sum_c x[r, c] * (q[e, m, c] - 8) * scales[e, m, c // G] for the rows
    r of expert e (``offsets`` of ``dispatch``, or of some of its experts, at a 16-byte
    aligned address; None with one matrix: every row); zeros for rows that no expert owns.

    x [N, C] bf16, packed [E, M, C/2] uint8 (even c in the low four bits), scales
    [E, M, C/G] bf16 with G = 32, 64 or 128. See latent_tail_expert_matvec4 and
    ``quantize4``."""
    N, C = _shape(x, "x", 2)
    i = _index(x, "x")
    E, M, _ = _shape(packed, "packed", 3)
    groups = _shape(scales, "scales", 3)[2]
    if groups == 0 or C % groups != 0:
        raise ValueError(f"scales: {groups} groups do not divide {C} columns")
    if out is None:
        out = _empty((N, M), _BF16, i, stream)
    _call("latent_tail_expert_matvec4", i, stream, _ptr(x, "x", _BF16, (N, C), i),
          _ptr(packed, "packed", _U8, (E, M, C // 2), i),
          _ptr(scales, "scales", _BF16, (E, M, groups), i),
          _ptr(offsets, "offsets", _I32, (E + 1,), i), _ptr(out, "out", _BF16, (N, M), i),
          N, E, M, C, C // groups)
    return out


def quantize4(weights, group: int):
    """(packed, scales) of ``weights`` [E, M, C] (or [M, C]: one matrix) for
    ``expert_matvec4``: per group of columns scale = max|w| / 7, rounded to bf16, and
    q = round(w / scale) + 8 in [0, 15]. Plain torch operations, done once per weight."""
    if weights.dim() == 2:
        weights = weights[None]
    w = weights.float().unflatten(-1, (-1, group))
    scales = (w.abs().amax(-1) / 7.0).to(_BF16)
    step = scales.float()[..., None]
    q = torch.where(step > 0, torch.round(w / step), torch.zeros_like(w))
    q = (q.clamp(-8, 7) + 8).to(_U8).flatten(-2)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous(), scales.contiguous()


def _gate_kind(gate, T, H):
    """Kind, dtype and shape of a gate: None, [T, 1] or [H] fp32, [T, H] bf16."""
    if gate is None:
        return _GATE_NONE, None, None
    if not isinstance(gate, torch.Tensor):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dim() == 1:
        return _GATE_CHANNEL, _F32, (H,)
    if gate.dim() == 2 and gate.shape[1] == 1:
        return _GATE_TOKEN, _F32, (T, 1)
    return _GATE_FULL, _BF16, (T, H)


def _residual_type(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is _BF16:
        return 0
    if t.dtype is _F32:
        return 1
    raise TypeError(f"{name}: expected torch.bfloat16 or torch.float32, got {t.dtype}")


def residual_norm(block, residual, post_weight, next_weight, eps: float, gate=None,
                  residual_scale: float = 1.0, residual_out=None, next_out=None, stream=None):
    """(residual_out, next_out) with
    residual_out = residual_scale * residual + gate * rms_norm(block, post_weight) and
    next_out = rms_norm(residual_out, next_weight).

    block [T, H] bf16, residual [T, H] bf16 or fp32, weights [H] fp32 or None (that
    norm is left out; next_out is then None), gate None, [T, 1] fp32, [H] fp32 or
    [T, H] bf16. residual_out may be residual itself. See latent_tail_residual_norm."""
    T, H = _shape(block, "block", 2)
    i = _index(block, "block")
    kind, gate_dtype, gate_shape = _gate_kind(gate, T, H)
    f32 = _residual_type(residual, "residual")
    if residual_out is None:
        residual_out = _empty((T, H), residual.dtype, i, stream)
    if next_out is None and next_weight is not None:
        next_out = _empty((T, H), _BF16, i, stream)
    _call("latent_tail_residual_norm", i, stream, _ptr(block, "block", _BF16, (T, H), i),
          _ptr(residual, "residual", residual.dtype, (T, H), i),
          _ptr(post_weight, "post_weight", _F32, (H,), i),
          _ptr(gate, "gate", gate_dtype, gate_shape, i),
          _ptr(next_weight, "next_weight", _F32, (H,), i),
          _ptr(residual_out, "residual_out", residual.dtype, (T, H), i),
          _ptr(next_out, "next_out", _BF16, (T, H), i), T, H, kind, f32, residual_scale, eps)
    return residual_out, next_out


@functools.lru_cache(maxsize=256)
def residual_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(load_library().latent_tail_residual_norm_backward_workspace_size(T, H))


def residual_norm_backward(grad_residual_out, grad_next, block, residual_out, post_weight,
                           next_weight, eps: float, gate=None, residual_scale: float = 1.0,
                           workspace=None, stream=None):
    """(grad_block, grad_residual, grad_post_weight, grad_gate, grad_next_weight) of
    ``residual_norm`` (None for what was not given), from the gradients of its outputs
    and its stored residual_out. grad_residual_out may be None (zero) where grad_next is
    given; grad_next is given exactly when next_weight is. See
    latent_tail_residual_norm_backward."""
    T, H = _shape(block, "block", 2)
    i = _index(block, "block")
    kind, gate_dtype, gate_shape = _gate_kind(gate, T, H)
    f32 = _residual_type(residual_out, "residual_out")
    rdt = residual_out.dtype
    given = (_ptr(grad_residual_out, "grad_residual_out", rdt, (T, H), i),
             _ptr(grad_next, "grad_next", _BF16, (T, H), i),
             _ptr(block, "block", _BF16, (T, H), i),
             _ptr(residual_out, "residual_out", rdt, (T, H), i),
             _ptr(post_weight, "post_weight", _F32, (H,), i),
             _ptr(gate, "gate", gate_dtype, gate_shape, i),
             _ptr(next_weight, "next_weight", _F32, (H,), i))
    grad_block, grad_residual = _like(block, stream), _like(residual_out, stream)
    grad_post = None if post_weight is None else _like(post_weight, stream)
    grad_gate = None if gate is None else _like(gate, stream)
    grad_nextw = None if next_weight is None else _like(next_weight, stream)
    if workspace is None:
        ws_bytes = max(16, residual_norm_backward_workspace_size(T, H))
        workspace = _empty((ws_bytes,), _U8, i, stream)
        ws = workspace.data_ptr()
    else:
        ws, ws_bytes = _workspace(workspace, i)
    _call("latent_tail_residual_norm_backward", i, stream, *given, grad_block.data_ptr(),
          grad_residual.data_ptr(), 0 if grad_post is None else grad_post.data_ptr(),
          0 if grad_gate is None else grad_gate.data_ptr(),
          0 if grad_nextw is None else grad_nextw.data_ptr(),
          T, H, kind, f32, residual_scale, eps, ws, ws_bytes)
    return grad_block, grad_residual, grad_post, grad_gate, grad_nextw
