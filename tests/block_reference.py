"""Plain 64-bit forms of the operators around the tail, and the bounds their
results are held to (test infrastructure; no CUDA kernels of this repository).

Bounds. U32 = 2^-24 and UBF = 2^-8 are the unit roundoffs of FP32 (24-bit significand) and
bf16 (8-bit significand). A
bf16 output that is rounded once from an FP32 value f with |f - ref| <= e differs
from ref by at most e + UBF * (|ref| + e). The FP32 error e of a sum of n
products is at most (n + 2) * U32 * sum |products| for any order of summation;
where the kernels' order is a tree, CHAIN = 256 roundings cover the longest chain
(H <= 16384: 16 products per thread, 5 + 32 additions over lanes and warps) with
the square root, division and factors applied afterwards.
"""

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8
CHAIN = 256


def bf16_bound(ref, err32):
    return err32 + UBF * (ref.abs() + err32)


def assert_within(got, ref, bound, what=""):
    got = got.double()
    assert got.shape == ref.shape, what
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    diff = torch.where(nan | (got == ref), torch.zeros_like(ref), (got - ref).abs())
    bad = ~(diff <= bound) & ~nan & (got != ref)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got "
            f"{got.reshape(-1)[i].item()!r}, want {ref.reshape(-1)[i].item()!r}, bound "
            f"{torch.as_tensor(bound).expand_as(ref).reshape(-1)[i].item():.3g}")


def dispatch(ids, E):
    """(order, position, offsets) by a Python sort."""
    flat = ids.cpu().reshape(-1).tolist()
    key = [v if 0 <= v < E else E for v in flat]
    order = sorted(range(len(flat)), key=lambda i: (key[i], i))
    position = [0] * len(flat)
    for r, i in enumerate(order):
        position[i] = r if key[i] < E else -1 - r
    offsets = [sum(k < e for k in key) for e in range(E + 1)] if len(flat) < 4096 else \
        torch.searchsorted(torch.tensor(sorted(key)), torch.arange(E + 1)).tolist()
    as32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return as32(order), as32(position).reshape(ids.shape), as32(offsets)


def combine(rows, position, weights):
    """(out, sum of |products|) in float64."""
    T, K = position.shape
    out = torch.zeros(T, rows.shape[1], dtype=torch.float64, device=rows.device)
    mag = torch.zeros_like(out)
    for k in range(K):
        p = position[:, k].long()
        t = torch.nonzero((p >= 0) & (p < T * K)).reshape(-1)
        term = rows[p[t]].double()
        if weights is not None:
            term = term * weights[t, k].double()[:, None]
        out[t] += term
        mag[t] += term.abs()
    return out, mag


def combine_backward(grad_out, rows, position, weights):
    """(grad_rows, grad_weights, sum of |products| of grad_weights) in float64."""
    T, K = position.shape
    g = grad_out.double()
    grad_rows = torch.zeros(T * K, g.shape[1], dtype=torch.float64, device=g.device)
    gw = torch.zeros(T, K, dtype=torch.float64, device=g.device)
    mag = torch.zeros_like(gw)
    for k in range(K):
        p = position[:, k].long()
        t = torch.nonzero((p >= 0) & (p < T * K)).reshape(-1)
        w = torch.ones(len(t), 1, dtype=torch.float64, device=g.device) if weights is None \
            else weights[t, k].double()[:, None]
        grad_rows[p[t]] = w * g[t]
        if rows is not None:
            prod = g[t] * rows[p[t]].double()
            gw[t, k] = prod.sum(1)
            mag[t, k] = prod.abs().sum(1)
    return grad_rows, gw, mag


def unpack4(packed, scales):
    """[E, M, C] float64 weights."""
    q = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2).double() - 8
    G = q.shape[-1] // scales.shape[-1]
    return q * scales.double().repeat_interleave(G, dim=-1)


def matvec4(x, packed, scales, offsets):
    """(out, sum of |products|) in float64."""
    N, M, E = x.shape[0], packed.shape[1], packed.shape[0]
    bounds = [0, N] if offsets is None else offsets.tolist()
    out = torch.zeros(N, M, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e in range(E):
        a, b = bounds[e], bounds[e + 1]
        if a < b:
            w = unpack4(packed[e:e + 1], scales[e:e + 1])[0]
            out[a:b] = x[a:b].double() @ w.t()
            mag[a:b] = x[a:b].double().abs() @ w.t().abs()
    return out, mag


def rms(v, w, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w


def residual_norm(block, residual, post, gate, nxt, scale, eps):
    """(v, z) in the inputs' type (call with float64)."""
    u = block if post is None else rms(block, post, eps)
    v = scale * residual + (u if gate is None else gate * u)
    return v, None if nxt is None else rms(v, nxt, eps)
