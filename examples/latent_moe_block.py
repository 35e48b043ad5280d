"""A latent-MoE block around the output tail, for decoding and for training.

Decode step (``DecodeBlock``): the router's choices are sorted by expert, the experts
run on 4-bit weights (gate/up and down projections), their rows come back weighted as
the tail's routed operand, the tail projects them up and adds the shared output, and
one kernel applies the norm after the block, its gate, the residual sum and the next
block's norm. All buffers are kept, so the step can be captured in a CUDA graph.

Training step (``train_step``): the same block with bf16 experts, through the autograd
wrappers for dispatch, combine and the norms.

    python examples/latent_moe_block.py            # both, on small shapes
"""

from __future__ import annotations

import math
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta

EPS = 1e-6


def make_weights(L, F, H, E, seed, device="cuda"):
    """Random weights: experts [E, 2F, L] and [E, L, F], up-projection [H, L], norms."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    bf16 = torch.bfloat16

    def normal(*shape, scale):
        return (torch.randn(*shape, generator=g, device=device) * scale).to(bf16)

    def norm(n):
        return 1.0 + 0.1 * torch.randn(n, generator=g, device=device)

    return dict(up=normal(E, 2 * F, L, scale=1 / math.sqrt(L)),
                down=normal(E, L, F, scale=1 / math.sqrt(F)),
                W=normal(H, L, scale=1 / math.sqrt(L)), latent_norm=norm(L), post=norm(H),
                next=norm(H), gate=0.5 + 0.1 * torch.randn(H, generator=g, device=device))


class DecodeBlock:
    """One block's decode step for T tokens with K choices among E experts."""

    def __init__(self, weights, T, K, group=32):
        self.w = weights
        E, F2, L = weights["up"].shape
        H = weights["W"].shape[0]
        dev, bf16 = weights["W"].device, torch.bfloat16
        self.E, self.T, self.K = E, T, K
        self.up4 = lt.quantize4(weights["up"], group)
        self.down4 = lt.quantize4(weights["down"], group)

        def buffer(*shape, dtype=bf16):
            return torch.empty(*shape, dtype=dtype, device=dev)

        n, i32 = T * K, torch.int32
        self.dispatched = lt.Dispatched(buffer(n, L), buffer(E + 1, dtype=i32),
                                        buffer(n, dtype=i32), buffer(T, K, dtype=i32))
        self.sort_workspace = buffer(max(16, lt.dispatch_workspace_size(T, K, E)),
                                     dtype=torch.uint8)
        self.hidden, self.rows = buffer(n, F2), buffer(n, L)
        self.routed, self.out = buffer(1, T, L), buffer(T, H)
        self.workspace = buffer(max(256, lt.latent_tail_workspace_size(1, T, L, H)),
                                dtype=torch.uint8)
        self.next = buffer(T, H)

    def __call__(self, x, expert_ids, expert_weights, shared, residual):
        """x [T, L] latent tokens, expert_ids [T, K] int32, expert_weights [T, K] fp32,
        shared [1, T, H], residual [T, H] (updated in place). Returns (residual, the
        next block's normalized input)."""
        w, d = self.w, self.dispatched
        lt.dispatch(x, expert_ids, self.E, *d, workspace=self.sort_workspace)
        lt.expert_matvec4(d.rows, *self.up4, d.offsets, out=self.hidden)
        gate, up = self.hidden.chunk(2, dim=1)
        act = torch.nn.functional.silu(gate) * up
        lt.expert_matvec4(act, *self.down4, d.offsets, out=self.rows)
        lt.combine(self.rows, d.position, expert_weights, out=self.routed[0])
        lt.forward(self.routed, shared, w["latent_norm"], w["W"], EPS, out=self.out,
                   workspace=self.workspace)
        return lt.residual_norm(self.out, residual, w["post"], w["next"], EPS, gate=w["gate"],
                                residual_out=residual, next_out=self.next)


def train_step(weights, x, expert_ids, expert_weights, shared, residual, residual_scale=1.0):
    """The block with bf16 experts under autograd (the tail in torch operations: its
    kernels have no backward pass). Returns (residual, next input)."""
    w = weights
    E, F2, L = w["up"].shape
    d = lta.dispatch_rows(x, expert_ids, E)
    parts = []
    bounds = d.offsets.tolist()
    for e in range(E):
        rows = d.rows[bounds[e]:bounds[e + 1]]
        gate, up = (rows @ w["up"][e].t()).chunk(2, dim=1)
        parts.append((torch.nn.functional.silu(gate) * up) @ w["down"][e].t())
    parts.append(d.rows[bounds[E]:])  # choices without an expert: zero rows
    routed = lta.combine_rows(torch.cat(parts), d.position, expert_weights).float()
    latent = routed * torch.rsqrt(routed.square().mean(-1, keepdim=True) + EPS) * w["latent_norm"]
    out = latent.to(torch.bfloat16) @ w["W"].t() + shared
    return lta.residual_norm(out, residual, w["post"], w["next"], EPS, gate=w["gate"],
                             residual_scale=residual_scale)


def inputs(T, K, L, H, E, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device=device)
    top = logits.topk(K, dim=1)
    bf16 = torch.bfloat16
    return (torch.randn(T, L, generator=g, device=device).to(bf16), top.indices.to(torch.int32),
            torch.softmax(top.values, dim=1),
            torch.randn(1, T, H, generator=g, device=device).to(bf16),
            torch.randn(T, H, generator=g, device=device).to(bf16))


def main():
    T, K, L, F, H, E = 16, 4, 256, 128, 512, 32
    w = make_weights(L, F, H, E, seed=0)
    x, ids, ew, shared, residual = inputs(T, K, L, H, E, seed=1)
    step = DecodeBlock(w, T, K)
    step(x, ids, ew, shared, residual.clone())  # first call sets the kernels up
    graph, r = torch.cuda.CUDAGraph(), residual.clone()
    with torch.cuda.graph(graph):
        out, nxt = step(x, ids, ew, shared, r)
    graph.replay()
    lt.latent_tail_check()
    print("decode: residual", tuple(out.shape), "next", tuple(nxt.shape),
          "rms of next %.3f" % nxt.float().square().mean().sqrt().item())

    params = {k: v.clone().requires_grad_(True) for k, v in w.items()}
    xt = x.clone().requires_grad_(True)
    out, nxt = train_step(params, xt, ids, ew, shared[0], residual)
    (out.float().square().mean() + nxt.float().square().mean()).backward()
    print("train: |grad x| %.3g, |grad up| %.3g, |grad gate| %.3g" % (
        xt.grad.float().norm(), params["up"].grad.float().norm(), params["gate"].grad.norm()))


if __name__ == "__main__":
    main()
