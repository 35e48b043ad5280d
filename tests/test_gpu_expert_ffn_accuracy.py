"""How far the gradients of the gated block and of the example's training step are from
those in 64 bits, as a whole and in slices of 16 columns, for each way of keeping the
projections.

Expected errors, as a share of a gradient's norm. Rounding to bf16 is off by at most
UBF |v|, evenly distributed, so by UBF / sqrt(3) of the norm at most; independent roundings
add in squares. Six lie on the way of each gradient (g, u, h or dg and du, dh, the result,
and one more where the sum is of rounded terms): sqrt(6 / 3) UBF = 1.4 UBF. An error of g
enters a'(g) and a(g) by at most 1.3 times its share for normal gates. A value kept in 8 bits
is off by a unit over sqrt(12) and a unit is at most 1/63.75 of the largest of 16 values,
2.13 times their root mean square for normal ones: K8 = 2.13 / (63.75 sqrt(12)) = 0.0097;
g and u both enter, g by 1.3: sqrt(1 + 1.3^2) K8. With x kept in 8 bits too the gradient of up
has another K8.
Norms of many elements lie within a few percent of that, those of slices of 16 columns within
half as much again."""

import importlib.util
import math
from pathlib import Path

import pytest
import torch

from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300.binding import latent_tail_check

import block_reference as br
import experts_reference as er
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
K8 = 2.13 / (63.75 * math.sqrt(12))
OF_BF16 = 1.3 * math.sqrt(2) * br.UBF
OF_8BIT = math.hypot(OF_BF16, math.sqrt(1 + 1.3 ** 2) * K8)
OF_8BIT_X = math.hypot(OF_8BIT, K8)
# of x, up and down
TOLERANCE = {"bf16": (OF_BF16,) * 3, "8bit": (OF_8BIT,) * 3,
             "all8bit": (OF_8BIT, OF_8BIT_X, OF_8BIT)}

_spec = importlib.util.spec_from_file_location(
    "latent_moe_block_accuracy",
    Path(__file__).resolve().parents[1] / "examples" / "latent_moe_block.py")
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def slices_off(got, want):
    """The worst of the slices of 16 columns, and of 16 rows of each matrix, that have half the
    mean norm of one."""
    worst = 0.0
    for dim in (-1, -2):
        if want.dim() < 3 and dim == -2:
            continue
        a, b = (t.double().split(16, dim=dim) for t in (got, want))
        typical = want.norm() / math.sqrt(len(b))
        for s, t in zip(a, b):
            if t.shape[dim] == 16 and t.norm() >= 0.5 * typical:
                worst = max(worst, off(s, t))
    return worst


def ffn_in_64_bits(x, up, down, offsets, act):
    out = torch.zeros(x.shape[0], down.shape[1], dtype=torch.float64, device=x.device)
    for e, (a, b) in enumerate(er.bounds(offsets, x.shape[0], up.shape[0])):
        if a < b:
            gate, u = (x[a:b] @ up[e].t()).chunk(2, dim=1)
            out[a:b] = (er.act(gate, act) * u) @ down[e].t()
    return out


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "8bit", "all8bit"])
@pytest.mark.parametrize("N,C,F,M,counts", [(512, 512, 256, 512, None),
                                            (1000, 264, 136, 200, (300, 0, 77, 600))])
def test_gradients_of_the_gated_block(N, C, F, M, counts, save, act):
    E = 1 if counts is None else len(counts)
    offsets = None if counts is None else torch.tensor(
        [sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(N)
    new = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(  # noqa: E731
        BF16).requires_grad_(True)
    leaves = new(N, C), new(E, 2 * F, C, scale=C ** -0.5), new(E, M, F, scale=F ** -0.5)
    dy = torch.randn(N, M, generator=g, device="cuda").to(BF16)
    lta.expert_ffn(*leaves, offsets, activation=act, save=save).backward(dy)
    latent_tail_check()
    wide = [t.detach().double().requires_grad_(True) for t in leaves]
    ffn_in_64_bits(*wide, offsets, act).backward(dy.double())
    for name, got, ref, tolerance in zip(("x", "up", "down"), leaves, wide, TOLERANCE[save]):
        whole, part = off(got.grad, ref.grad), slices_off(got.grad, ref.grad)
        assert whole <= tolerance, name
        assert part <= 1.5 * tolerance, name
        assert not got.grad[ref.grad == 0].any()


def train_step_in_64_bits(w, x, ids, ew, shared, residual, scale):
    eps = example.EPS
    routed = torch.zeros_like(x)
    for k in range(ids.shape[1]):
        for e in range(w["up"].shape[0]):
            t = torch.nonzero(ids[:, k] == e).reshape(-1)
            if len(t):
                gate, u = (x[t] @ w["up"][e].t()).chunk(2, dim=1)
                y = (er.act(gate, "silu") * u) @ w["down"][e].t()
                routed = routed.index_add(0, t, ew[t, k, None] * y)
    out = br.rms(routed, w["latent_norm"], eps) @ w["W"].t() + shared
    return br.residual_norm(out, residual, w["post"], w["gate"], w["next"], scale, eps)


def test_the_example_s_training_step():
    """Residual, next input and every gradient, for each way of keeping the projections.

    On the way from the results back to the experts lie, besides the block's six, roundings of
    the norms' gradient, of the tail's product and its gradient, of combine, dispatch and
    their gradients: twelve in all, 2 UBF, which the norms' gradients may raise by half. The
    other parameters' gradients do not depend on what is kept: the same bits."""
    T, K, L, F, H, E = 256, 4, 256, 128, 512, 8
    weights = example.make_weights(L, F, H, E, seed=3)
    x, ids, ew, shared, residual = example.inputs(T, K, L, H, E, seed=4)
    ids[5, 1] = ids[100, 0] = -1
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    dout, dnext = (torch.randn(T, H, generator=g, device="cuda").to(BF16) for _ in range(2))

    def leaves(double):
        own = dict(weights, x=x, ew=ew, shared=shared[0], residual=residual)
        return {k: (v.double() if double else v.clone()).requires_grad_(True)
                for k, v in own.items()}

    wide = leaves(True)
    want = train_step_in_64_bits(wide, wide["x"], ids, wide["ew"], wide["shared"],
                                 wide["residual"], 0.5)
    torch.autograd.backward(want, (dout.double(), dnext.double()))
    tolerance = {"bf16": 3 * br.UBF, "8bit": math.hypot(3 * br.UBF, OF_8BIT)}
    tolerance["all8bit"] = math.hypot(tolerance["8bit"], K8)
    first = None
    for save in ("bf16", "8bit", "all8bit"):
        own = leaves(False)
        got = example.train_step(own, own["x"], ids, own["ew"], own["shared"], own["residual"],
                                 residual_scale=0.5, save=save)
        torch.autograd.backward(got, (dout, dnext))
        latent_tail_check()
        for a, b in zip(got, want):
            assert off(a.detach(), b.detach()) <= 3 * br.UBF
        for k, v in own.items():
            limit = tolerance[save] if k in ("x", "up", "down") else tolerance["bf16"]
            assert off(v.grad, wide[k].grad) <= limit, (save, k)
        if first is None:
            first = got, own
        else:
            assert all(torch.equal(a, b) for a, b in zip(got, first[0]))
            for k in ("W", "latent_norm", "post", "next", "gate", "shared", "residual", "ew"):
                assert torch.equal(own[k].grad, first[1][k].grad), (save, k)
