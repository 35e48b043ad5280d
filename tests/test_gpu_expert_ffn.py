"""The gated block with its gradients through torch.autograd, the block with dispatch and
combine around it, and the workloads of perf/more_operators.py against their definitions."""

import importlib.util
from pathlib import Path

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300.binding import latent_tail_check

import block_reference as br
import experts_reference as er
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

_spec = importlib.util.spec_from_file_location(
    "more_operator_workloads", Path(__file__).resolve().parents[1] / "perf" / "more_operators.py")
workloads = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(workloads)
CASES = [c for c in workloads.listed() if c["T"] <= 1024]


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def leaves(N, C, F, M, E, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(  # noqa: E731
        BF16).requires_grad_(True)
    return (new(N, C), new(E, 2 * F, C, scale=C ** -0.5), new(E, M, F, scale=F ** -0.5),
            torch.randn(N, M, generator=g, device="cuda").to(BF16))


def exact_ffn(x, up, down, offsets, act):
    out = torch.zeros(x.shape[0], down.shape[1], dtype=torch.float64, device=x.device)
    for e, (a, b) in enumerate(er.bounds(offsets, x.shape[0], up.shape[0])):
        if a < b:
            gate, u = (x[a:b] @ up[e].t()).chunk(2, dim=1)
            out[a:b] = (er.act(gate, act) * u) @ down[e].t()
    return out


# Norm of a gradient's error over its norm. bf16: the values between the ends are rounded
# at g, u, h, dh, dg or du, and the result, six of 2^-8 at most each. 8 bits: a kept value is
# off by at most 1/127 of its group's largest magnitude, which for normal values is under
# three times their root mean square: 3/127 of g, of u, and, where x is kept so too, of x.
TOLERANCE = {"bf16": 6 * br.UBF, "8bit": 6 * br.UBF + 2 * 3 / 127,
             "all8bit": 6 * br.UBF + 3 * 3 / 127}


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "8bit", "all8bit"])
@pytest.mark.parametrize("N,C,F,M,counts", [(40, 72, 24, 56, None), (300, 264, 136, 200,
                                                                     (100, 0, 7, 180))])
def test_expert_ffn(N, C, F, M, counts, save, act):
    E = 1 if counts is None else len(counts)
    offsets = None if counts is None else torch.tensor(
        [sum(counts[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    x, up, down, dy = leaves(N, C, F, M, E, seed=N)
    out = lta.expert_ffn(x, up, down, offsets, activation=act, save=save)
    out.backward(dy)
    latent_tail_check()
    wide = [t.detach().double().requires_grad_(True) for t in (x, up, down)]
    want = exact_ffn(*wide, offsets, act)
    want.backward(dy.double())
    assert (out.detach().double() - want.detach()).norm() <= 3 * br.UBF * want.detach().norm()
    for got, ref in zip((x, up, down), wide):
        assert got.grad.dtype == BF16
        assert (got.grad.double() - ref.grad).norm() <= TOLERANCE[save] * ref.grad.norm()
        assert torch.equal(got.grad[ref.grad == 0], torch.zeros_like(got.grad[ref.grad == 0]))


@pytest.mark.parametrize("wanted", [(True, False, False), (False, True, False),
                                    (False, False, True), (True, False, True),
                                    (False, False, False)])
def test_expert_ffn_of_some_gradients(wanted):
    """A gradient that is not wanted is not computed; the others have the same bits."""
    N, C, F, M, E = 40, 72, 24, 56, 1
    full = leaves(N, C, F, M, E, seed=1)
    lta.expert_ffn(*full[:3]).backward(full[3])
    some = leaves(N, C, F, M, E, seed=1)
    for t, w in zip(some, wanted):
        t.requires_grad_(w)
    out = lta.expert_ffn(*some[:3])
    assert out.requires_grad == any(wanted)
    if any(wanted):
        out.backward(some[3])
    for a, b, w in zip(some, full, wanted):
        assert (a.grad is not None) == w
        if w:
            assert torch.equal(a.grad, b.grad)


def test_expert_ffn_takes_strided_gradients():
    N, C, F, M, E = 40, 72, 24, 56, 1
    a, b = (leaves(N, C, F, M, E, seed=2) for _ in range(2))
    lta.expert_ffn(*a[:3]).backward(a[3])
    wide = torch.zeros(N, 2 * M, dtype=BF16, device="cuda")
    wide[:, 1::2] = b[3]
    lta.expert_ffn(*b[:3]).backward(wide[:, 1::2])
    for s, t in zip(a[:3], b[:3]):
        assert torch.equal(s.grad, t.grad)


def test_block_of_dispatch_experts_and_combine():
    """Tokens to experts and back, forward and backward, against the same sum per token."""
    T, K, E, C, F = 70, 3, 8, 136, 40
    x, up, down, dy = leaves(T, C, F, C, E, seed=4)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    ids = torch.randn(T, E, generator=g, device="cuda").topk(K).indices.to(torch.int32)
    ids[3, 1] = ids[9, 0] = -1
    weights = torch.rand(T, K, generator=g, device="cuda").requires_grad_(True)
    d = lta.dispatch_rows(x, ids, E)
    out = lta.combine_rows(lta.expert_ffn(d.rows, up, down, d.offsets, save="bf16"), d.position,
                           weights)
    out.backward(dy)
    latent_tail_check()
    wx, wup, wdown, ww = (t.detach().double().requires_grad_(True) for t in (x, up, down, weights))
    want = torch.zeros(T, C, dtype=torch.float64, device="cuda")
    for k in range(K):
        for e in range(E):
            t = torch.nonzero(ids[:, k] == e).reshape(-1)
            if len(t):
                gate, u = (wx[t] @ wup[e].t()).chunk(2, dim=1)
                want = want.index_add(0, t, ww[t, k, None] * ((er.act(gate, "silu") * u)
                                                              @ wdown[e].t()))
    want.backward(dy.double())
    # (dispatch and combine round once more on each side)
    assert (out.detach().double() - want.detach()).norm() <= 4 * br.UBF * want.detach().norm()
    for got, ref in ((x, wx), (up, wup), (down, wdown), (weights, ww)):
        assert (got.grad.double() - ref.grad).norm() <= 8 * br.UBF * ref.grad.norm()


# ---------------------------------------------------------------- workloads
def parts(v):
    return list(v) if isinstance(v, (tuple, list)) else [v]


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c["name"] for c in CASES])
def test_workload_against_its_definition(case, own, monkeypatch):
    """Norm of the error over the norm of the exact value. Plain form and kernel round once to
    bf16, 2^-8 at most; gradients of a gated block also dg and du, and their terms' errors add
    up like the terms (independent roundings): 2 * 2^-8. FP32 sums are below that by far."""
    monkeypatch.setattr(workloads, "own", own)
    got = parts(workloads.run(workloads.prepare(case, 11)))
    want = parts(workloads.exact(case, 11))
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert (a.double() - b).norm() <= 2 * br.UBF * b.norm()
