"""Plain 64-bit forms of the bf16 experts, their gradients and the 8-bit form of kept
activations (test infrastructure; no CUDA kernels of this repository)."""

import math

import torch

GROUP = 16


def power2(n):
    """2^n in 64 bits, exactly (exp2 on the GPU may be off in its last bit)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def bounds(offsets, N, E):
    """Rows [a, b) of each expert: offsets cut to [0, N] and to their running maximum."""
    if offsets is None:
        return [(0, N)]
    got, top = [], 0
    for v in offsets.tolist():
        top = max(top, min(max(v, 0), N))
        got.append(top)
    return list(zip(got[:-1], got[1:]))


def matmul(x, weights, offsets):
    """(out, sum of |products|) in float64."""
    N, (E, M, _) = x.shape[0], weights.shape
    out = torch.zeros(N, M, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e, (a, b) in enumerate(bounds(offsets, N, E)):
        if a < b:
            w = weights[e].double().t()
            out[a:b] = x[a:b].double() @ w
            mag[a:b] = x[a:b].double().abs() @ w.abs()
    return out, mag


def matmul_backward(grad, x, weights, offsets):
    """(grad_x, grad_weights) in float64."""
    N, (E, M, C) = x.shape[0], weights.shape
    gx = torch.zeros(N, C, dtype=torch.float64, device=x.device)
    gw = torch.zeros(E, M, C, dtype=torch.float64, device=x.device)
    for e, (a, b) in enumerate(bounds(offsets, N, E)):
        if a < b:
            g = grad[a:b].double()
            gx[a:b] = g @ weights[e].double()
            gw[e] = g.t() @ x[a:b].double()
    return gx, gw


def owned(offsets, N, E, device):
    """Whether an expert owns the row."""
    mask = torch.zeros(N, dtype=torch.bool, device=device)
    for a, b in bounds(offsets, N, E):
        mask[a:b] = True
    return mask


def act_argument(g, name):
    """s with a(g) = g sigmoid(s): 0.5 (1 + tanh(y)) = sigmoid(2 y), without the sum's
    cancellation far out on the negative side."""
    return g if name == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)


def act(g, name):
    return g * torch.sigmoid(act_argument(g, name))


def quantize8(v):
    """(values, exponents) of ``v`` [..., C] (float64) from the definition: the least e >= 1
    for which the largest magnitude of the group rounds to at most 127 units."""
    C = v.shape[-1]
    part = torch.nn.functional.pad(v, (0, -C % GROUP)).unflatten(-1, (-1, GROUP))
    top = part.abs().amax(-1)
    bad = ~torch.isfinite(part).all(-1)
    top = torch.where(bad, torch.ones_like(top), top)

    def fits(e):
        return torch.round(top * power2(127 - e)) <= 127

    e = (torch.frexp(top)[1] + 127 - 12).clamp(min=1).long()
    assert not (fits(e - 1) & (e > 1) & (top > 0)).any()  # below the least
    for _ in range(8):
        e = torch.where(fits(e), e, e + 1)
    assert fits(e).all()
    zero = (top == 0) | bad
    n = torch.round(part * power2(127 - e)[..., None])
    q = torch.where(zero[..., None], torch.zeros_like(n), n).to(torch.int8)
    e8 = torch.where(bad, 255, torch.where(top == 0, 0, e)).to(torch.uint8)
    return q.flatten(-2)[..., :C].contiguous(), e8


def dequantize8(values, exponents):
    """float64 values of an 8-bit checkpoint."""
    e = exponents.long().repeat_interleave(GROUP, dim=-1)[..., :values.shape[-1]]
    v = values.double() * power2(e - 127)
    v = torch.where(e == 0, torch.zeros_like(v), v)
    return torch.where(e == 255, torch.full_like(v, math.nan), v)
