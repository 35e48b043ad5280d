"""The experts' operators at the edges of what the documentation allows."""

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


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "8bit"])
def test_gradient_where_the_gate_is_off_and_the_rest_is_large(act, save):
    """dg = dh u a'(g) is 0 where a'(g) is, also where dh u alone passes FP32's range. The
    gradient of a gate is read through a weight of 1: dx = dg exactly.

    FP32 error of dg: two products (2^-23 in all) and that of a', which is at most 2^-17 of
    |s| + |g s'| <= 1.2 + |g| here (|s| <= 30 where a' is not 0 in FP32), then one rounding of
    2^-8 to bf16 and another of the product."""
    gates = [-300.0, -200.0, -150.0, -2.0, 0.0, 0.5, 3.0, 150.0]
    large = [(1e30, 1e30), (3e38, 2.0), (-1e25, 1e20), (1e38, -1e38), (1e-3, 3e38), (2.0, 3.0)]
    rows = [(g, d, u) for g in gates for d, u in large]
    N, F, C = len(rows), 8, 8
    t = torch.tensor(rows, device="cuda").to(BF16)
    kept = torch.zeros(N, 2, F, dtype=BF16, device="cuda")
    kept[:, 0], kept[:, 1] = t[:, :1], t[:, 2:]
    saved = kept if save == "bf16" else lt.quantize8(kept)
    wide = (kept if save == "bf16" else lt.dequantize8(saved)).double()
    dh = t[:, 1:2].expand(N, F).contiguous()
    w = torch.zeros(1, 2 * F, C, dtype=BF16, device="cuda")
    w[0, :F] = torch.eye(F)
    # du is multiplied by weights of 0: it has to be finite for dx to be dg
    gate, up = wide[:, 0], wide[:, 1]
    s = torch.sigmoid(er.act_argument(gate, act))
    slope = torch.where(gate.abs() >= 150, (gate > 0).double(), s + gate * s * (1 - s) * (
        1 if act == "silu" else er.act_argument(torch.ones_like(gate), act) / 1.044715
        * (1 + 3 * 0.044715 * gate ** 2)))
    want, du = dh.double() * up * slope, dh.double() * gate * s
    most = torch.finfo(BF16).max
    ok = (want.abs() < most) & (du.abs() < most)
    assert ok[:len(large) * 3].all()
    gx, _, _ = lt.expert_gated_backward(dh, None, w, saved, activation=act)
    latent_tail_check()
    err = (dh.double() * up).abs() * (1.2 + gate.abs()) * 2.0 ** -17
    err = torch.where(gate.abs() >= 150, torch.zeros_like(err), err) + want.abs() * 2.0 ** -23
    bound = br.UBF * want.abs() + err * (1 + br.UBF)
    got = gx.double()
    assert torch.isfinite(got[ok]).all()
    assert ((got - want).abs() <= bound + br.UBF * (want.abs() + bound))[ok].all()


@pytest.mark.parametrize("N,M,C", [(65536, 512, 768), (65536, 256, 1920), (16377, 3840, 120)])
def test_sums_over_many_rows_that_four_pairs_share(N, M, C):
    """Integers whose sums stay below 2^24: exact, whatever the order."""
    g = torch.Generator(device="cuda")
    g.manual_seed(N + M)
    x, dy = (torch.randint(-3, 4, (N, n), generator=g, device="cuda").to(BF16) for n in (C, M))
    _, gw = lt.expert_matmul_backward(dy, x, None)
    latent_tail_check()
    assert torch.equal(gw[0], (dy.double().t() @ x.double()).to(BF16))


# --------------------------------------------------------------- under autograd
def ffn_leaves(N, C, F, M, E, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    new = lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(  # noqa: E731
        BF16).requires_grad_(True)
    return (new(N, C), new(E, 2 * F, C, scale=C ** -0.5), new(E, M, F, scale=F ** -0.5),
            torch.randn(N, M, generator=g, device="cuda").to(BF16))


@pytest.mark.parametrize("save", ["bf16", "8bit", "all8bit"])
def test_an_evaluation_pass_takes_no_memory_for_a_backward_pass(save):
    N, C, F, M = 4096, 256, 512, 256
    x, up, down, _ = ffn_leaves(N, C, F, M, 1, seed=1)
    want = lta.expert_ffn(x, up, down, save=save).detach()
    for mode in (torch.no_grad, torch.inference_mode):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        with mode():
            out = lta.expert_ffn(x, up, down, save=save)
        torch.cuda.synchronize()
        # hidden and out, in the allocator's pieces of 2 MB at most
        assert torch.cuda.max_memory_allocated() - before <= 2 * N * (F + M) + (4 << 20)
        assert torch.equal(out, want)


@pytest.mark.parametrize("reentrant", [False, True])
def test_under_activation_checkpointing(reentrant):
    """The first pass, without gradients in the one form, gives the same bits."""
    from torch.utils.checkpoint import checkpoint

    a, b = (ffn_leaves(300, 136, 72, 200, 1, seed=2) for _ in range(2))
    lta.expert_ffn(*a[:3], save="8bit").backward(a[3])
    out = checkpoint(lambda *t: lta.expert_ffn(*t, save="8bit"), *b[:3], use_reentrant=reentrant)
    out.backward(b[3])
    for s, t in zip(a[:3], b[:3]):
        assert torch.equal(s.grad, t.grad)
