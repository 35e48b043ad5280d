"""Host-side edges of the operators around the tail, on a machine without a GPU too."""

import weakref

import pytest
import torch

from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300 import binding
from latent_moe_output_gb300.binding import Status

# Fake, never-dereferenced addresses, 64 MiB apart.
BLOCK, RES, POST, GATE, NEXT, OUT, Z = (0x10000000 + 0x4000000 * i for i in range(7))


@pytest.fixture(scope="module")
def lib():
    from latent_moe_output_gb300 import build

    build.build()
    return binding.load_library()


# ------------------------------------------ in place: the residual alone
@pytest.mark.parametrize("T,H,rt", [(1, 64, 1), (2, 64, 0)])  # residual of a vector's bytes
@pytest.mark.parametrize("name", ["post", "gate", "next"])
def test_residual_out_on_a_vector_that_is_the_residual_too_is_refused(lib, T, H, rt, name):
    """residual_out may be exactly residual. Where a weight or a channel gate is that same
    array too, it would be read after it was written."""
    p = dict(post=POST, gate=GATE, next=NEXT)
    p[name] = RES
    st = lib.latent_tail_residual_norm(BLOCK, RES, p["post"], p["gate"], p["next"], RES, Z, T, H,
                                       2, rt, 1.0, 1e-6, None)
    assert st == Status.INVALID_ARG


# ------------------------------------------------ partial sums of the gradient
@pytest.mark.parametrize("H,per_sm", [(256, 2), (264, 1), (512, 1), (520, 6), (1024, 6), (7168, 1)])
def test_residual_norm_backward_has_a_partial_row_per_resident_cta(lib, H, per_sm):
    """... of the SMs that a size computed without a device allows for (304)."""
    got = lib.latent_tail_residual_norm_backward_workspace_size(1 << 20, H)
    assert got == 2 * 304 * per_sm * H * 4


# ------------------------------------------------- what a backward pass keeps
@pytest.fixture
def calls(monkeypatch):
    """The operators' calls by autograd, answered by torch operations on the CPU."""
    from latent_moe_output_gb300 import block

    seen = []

    def combine(rows, position, weights=None):
        seen.append("combine")
        got = rows[position.long()]
        return (got if weights is None else got * weights[..., None]).sum(1).to(rows.dtype)

    def combine_backward(grad_out, rows, position, weights=None):
        seen.append("combine_backward")
        T, K = position.shape
        grad_rows = torch.zeros(T * K, grad_out.shape[1], dtype=grad_out.dtype)
        term = grad_out[:, None].expand(-1, K, -1)
        grad_rows[position.reshape(-1).long()] = (
            term if weights is None else term * weights[..., None]).reshape(T * K, -1).to(
                grad_out.dtype)
        return grad_rows, None if rows is None else (rows[position.long()] * term).sum(-1).float()

    monkeypatch.setattr(block, "combine", combine)
    monkeypatch.setattr(block, "combine_backward", combine_backward)
    return seen


@pytest.mark.parametrize("weighted", [False, True])
def test_combine_without_a_gradient_of_the_weights_lets_go_of_the_rows(calls, weighted):
    """Only the gradient of the weights reads the rows: without it they may be written after
    the call, and are not kept alive for the backward pass."""
    rows = torch.randn(6, 8, dtype=torch.bfloat16)
    position = torch.arange(6, dtype=torch.int32).reshape(3, 2)
    weights = torch.full((3, 2), 0.5) if weighted else None
    leaf = rows.clone().requires_grad_(True)
    passed = leaf * 1
    kept = weakref.ref(passed)
    out = lta.combine_rows(passed, position, weights)
    with torch.no_grad():
        passed.mul_(2)
    del passed
    assert kept() is None
    out.float().sum().backward()
    assert torch.equal(leaf.grad, torch.full_like(rows, 0.5 if weighted else 1.0))
    assert calls == ["combine", "combine_backward"]


def test_combine_with_a_gradient_of_the_weights_keeps_the_rows(calls):
    rows = torch.randn(6, 8, dtype=torch.bfloat16)
    position = torch.arange(6, dtype=torch.int32).reshape(3, 2)
    weights = torch.full((3, 2), 0.5, requires_grad=True)
    changed = rows.clone()
    lta.combine_rows(rows, position, weights).float().sum().backward()
    assert torch.equal(weights.grad, rows[position.long()].sum(-1).float())
    out = lta.combine_rows(changed, position, weights)
    changed.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.float().sum().backward()


def test_gradients_at_any_offset_are_taken(calls, monkeypatch):
    """Autograd may pass a contiguous view that is not 16-byte aligned, e.g. of the gradient
    of flat tensors joined in one; the operators take aligned addresses alone."""
    from latent_moe_output_gb300 import block

    seen = []

    def aligned(call):
        def checked(*args, **kwargs):
            for t in args:
                if isinstance(t, torch.Tensor):
                    assert t.is_contiguous() and t.data_ptr() % 16 == 0
                    seen.append(t)
            return call(*args, **kwargs)
        return checked

    def norm(b, r, post, nxt, eps, gate=None, residual_scale=1.0):
        return b + r, (b + r) * 2

    def norm_backward(dv, dz, b, out, post, nxt, eps, gate=None, residual_scale=1.0):
        g = dv + 2 * dz
        return g, g, None, None, torch.zeros_like(nxt)

    def dispatch(x, ids, E):
        n = ids.numel()
        at = torch.arange(n, dtype=torch.int32)
        return block.Dispatched(x.repeat_interleave(ids.shape[1], 0), at[:E], at,
                                at.reshape(ids.shape))

    monkeypatch.setattr(block, "combine_backward", aligned(block.combine_backward))
    monkeypatch.setattr(block, "combine", aligned(block.combine))
    monkeypatch.setattr(block, "residual_norm", norm)
    monkeypatch.setattr(block, "residual_norm_backward", aligned(norm_backward))
    monkeypatch.setattr(block, "dispatch", dispatch)

    def flat(*tensors):  # a loss on one flat tensor with three values before the others
        start = torch.zeros(3, dtype=torch.bfloat16)
        joined = torch.cat([start] + [t.reshape(-1) for t in tensors])
        return (joined * joined.detach()).float().sum()

    new = lambda *s: torch.randn(*s, dtype=torch.bfloat16).requires_grad_(True)  # noqa: E731
    rows, x, b = new(6, 8), new(3, 8), new(2, 8)
    position = torch.arange(6, dtype=torch.int32).reshape(3, 2)
    flat(lta.combine_rows(rows, position)).backward()
    flat(lta.dispatch_rows(x, position, 4).rows).backward()
    flat(*lta.residual_norm(b, torch.zeros(2, 8, dtype=torch.bfloat16), None, torch.ones(8),
                            1e-6)).backward()
    assert len(seen) >= 8 and all(t.grad is not None for t in (rows, x, b))
