"""The operators around the tail used together: the example block's decode step
against a 64-bit form of the whole block, captured in a graph, and the autograd
wrappers against torch's gradients in 64 bits."""

import importlib.util
from pathlib import Path

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300.binding import latent_tail_check

import block_reference as br
import gpu_helpers as gh

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "latent_moe_block", Path(__file__).resolve().parents[1] / "examples" / "latent_moe_block.py")
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)
EPS = example.EPS


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def block_in_64_bits(step, x, ids, ew, shared, residual):
    w = step.w
    up, down = (br.unpack4(*q) for q in (step.up4, step.down4))
    routed = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = int(ids[t, k])
            if 0 <= e < step.E:
                gate, u = (up[e] @ x[t].double()).chunk(2)
                routed[t] += ew[t, k].double() * (down[e] @ (torch.sigmoid(gate) * gate * u))
    latent = br.rms(routed, w["latent_norm"].double(), EPS)
    out = latent @ w["W"].double().t() + shared[0].double()
    return br.residual_norm(out, residual.double(), w["post"].double(), w["gate"].double(),
                            w["next"].double(), 1.0, EPS)


@pytest.mark.parametrize("T,K,L,F,H,E", [(1, 4, 128, 64, 256, 8), (16, 4, 256, 128, 512, 32),
                                         (40, 2, 64, 96, 136, 5)])
def test_decode_block(T, K, L, F, H, E):
    w = example.make_weights(L, F, H, E, seed=T)
    x, ids, ew, shared, residual = example.inputs(T, K, L, H, E, seed=T + 1)
    if T > 1:
        ids[T // 2, 0] = -1  # a choice without an expert
    step = example.DecodeBlock(w, T, K)
    want_r, want_n = block_in_64_bits(step, x, ids, ew, shared, residual)
    r = residual.clone()
    out, nxt = step(x, ids, ew, shared, r)
    latent_tail_check()
    # the tolerance of the tail's own tests: several bf16 roundings lie between the ends
    for got, want in ((out, want_r), (nxt, want_n)):
        torch.testing.assert_close(got.double(), want, atol=gh.ATOL, rtol=gh.RTOL)
    graph, again = torch.cuda.CUDAGraph(), residual.clone()
    with torch.cuda.graph(graph):
        out2, nxt2 = step(x, ids, ew, shared, again)
    again.copy_(residual)
    first = (out.clone(), nxt.clone())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out2, first[0]) and torch.equal(nxt2, first[1])


def test_example_runs(capsys):
    example.main()
    text = capsys.readouterr().out
    assert "decode:" in text and "train:" in text


def test_autograd_dispatch_and_combine():
    T, K, E, L = 37, 4, 9, 136
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    x = torch.randn(T, L, generator=g, device="cuda").to(torch.bfloat16).requires_grad_(True)
    w = torch.rand(T, K, generator=g, device="cuda").requires_grad_(True)
    ids = torch.randint(-1, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    go = torch.randn(T, L, generator=g, device="cuda").to(torch.bfloat16)
    d = lta.dispatch_rows(x, ids, E)
    out = lta.combine_rows(d.rows, d.position, w)
    out.backward(go)
    # out[t] = x[t] * sum of its routed weights
    here = (ids >= 0)
    s = (w.detach().double() * here).sum(1, keepdim=True)
    br.assert_within(out.detach(), x.detach().double() * s,
                     br.bf16_bound(x.detach().double() * s, 6 * br.U32 * x.detach().abs() * s))
    # the rows' gradients are rounded to bf16 before they are summed: UBF per term
    gx = go.double() * s
    br.assert_within(x.grad, gx, 2 * br.UBF * gx.abs() + br.UBF * (1 + br.UBF) * gx.abs())
    gw = (go.double() * x.detach().double()).sum(1, keepdim=True) * here
    mag = (go.double() * x.detach().double()).abs().sum(1, keepdim=True)
    br.assert_within(w.grad, gw, br.CHAIN * br.U32 * mag.expand_as(gw))
    y = lta.combine_rows(d.rows.detach().requires_grad_(True), d.position)  # no weights
    y.sum().backward()


@pytest.mark.parametrize("use", ["both", "residual", "next"])
def test_autograd_residual_norm(use):
    T, H, scale = 9, 520, 0.5
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    new = lambda *s, dt=torch.float32: torch.randn(*s, generator=g, device="cuda").to(  # noqa: E731
        dt).requires_grad_(True)
    block, residual = new(T, H, dt=torch.bfloat16), new(T, H)
    post, nxt, gate = new(H), new(H), new(T, 1)
    args = (block, residual, post, nxt)
    v, z = lta.residual_norm(*args, EPS, gate=gate, residual_scale=scale)
    wide = [t.detach().double().requires_grad_(True) for t in (*args, gate)]
    wv, wz = br.residual_norm(wide[0], wide[1], wide[2], wide[4], wide[3], scale, EPS)
    dv, dz = torch.randn_like(v), torch.randn_like(z)
    loss, want = 0, 0
    if use != "next":
        loss, want = loss + (v * dv).sum(), want + (wv * dv.double()).sum()
    if use != "residual":
        loss = loss + (z.float() * dz.float()).sum()
        want = want + (wz * dz.double()).sum()
    loss.backward()
    want.backward()
    for got, ref in zip((*args, gate), wide):
        if ref.grad is None:
            continue
        tol = 2 * br.UBF if got.dtype == torch.bfloat16 else 1e-4
        scale_of = ref.grad.abs().max()
        assert (got.grad.double() - ref.grad).abs().max() <= tol * scale_of
