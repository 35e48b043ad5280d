"""The experts' operators at the edges of what the documentation allows."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300.binding import LatentTailError, Status, latent_tail_check

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


# ------------------------------------------------------ what the documentation says
def test_offsets_of_some_experts():
    """Experts 4 to 7 of a dispatch by a slice of its offsets, and 3 to 6 by a copy of one: the
    other experts' rows are zeros, and the slice that is not aligned is refused."""
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    counts = [5, 0, 9, 30, 2, 17, 0, 40, 11]
    offsets = torch.tensor([sum(counts[:i]) for i in range(10)], dtype=torch.int32, device="cuda")
    N, M, C = sum(counts), 72, 136
    x = torch.randint(-3, 4, (N, C), generator=g, device="cuda").to(BF16)
    w = torch.randint(-3, 4, (9, M, C), generator=g, device="cuda").to(BF16)
    whole = lt.expert_matmul(x, w, offsets)
    for first, of in ((4, offsets[4:9]), (3, offsets[3:8].clone())):
        a, b = sum(counts[:first]), sum(counts[:first + 4])
        out = lt.expert_matmul(x, w[first:first + 4], of)
        assert torch.equal(out[a:b], whole[a:b])
        assert not out[:a].any() and not out[b:].any()
    with pytest.raises(LatentTailError) as e:
        lt.expert_matmul(x, w[3:7], offsets[3:8])
    assert e.value.status == Status.ALIGNMENT


def test_bits_do_not_depend_on_the_offsets_or_on_what_is_kept():
    """The same rows and weights with other offsets around them, kept or not."""
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    N, E, F, C = 700, 3, 136, 712
    x = torch.randn(N, C, generator=g, device="cuda").to(BF16)
    w = (torch.randn(1, 2 * F, C, generator=g, device="cuda") * C ** -0.5).to(BF16)
    w = w.expand(E, 2 * F, C).contiguous()
    want = None
    for cuts in ((0, 700, 700, 700), (0, 1, 690, 700), (0, 0, 350, 700), (0, 256, 512, 700)):
        offsets = torch.tensor(cuts, dtype=torch.int32, device="cuda")
        for saved in (None, torch.empty(N, 2, F, dtype=BF16, device="cuda"),
                      lt.Checkpoint8.empty(N, 2, F)):
            hidden = lt.expert_gated(x, w, offsets, saved=saved)
            want = hidden if want is None else want
            assert torch.equal(hidden, want)


def test_largest_values_in_8_bits():
    """255/128 * 2^127 and the value below it, beside the largest, round to 64 units of 2^122:
    infinities when read back, as documented; everything below them is finite."""
    top = torch.tensor([0x7F7F, 0x7F7E, 0x7F7D, 0x7F00, 0x3F80], dtype=torch.int16).view(BF16)
    x = torch.zeros(2, 16, dtype=BF16)
    x[0, :5], x[1, 0], x[1, 1:4] = top, -top[1], top[2:]  # (with the largest, and without)
    kept = lt.quantize8(x.cuda())
    back = lt.dequantize8(kept).cpu()
    inf = float("inf")
    assert kept.exponents.tolist() == [[249], [248]]
    assert kept.values[0, :5].tolist() == [64, 64, 63, 32, 0]
    assert kept.values[1, :4].tolist() == [-127, 126, 64, 0]  # (126.5 units: to the even one)
    assert back[0, :5].tolist()[:2] == [inf, inf] and torch.isfinite(back[0, 2:]).all()
    assert torch.isfinite(back[1]).all()
    q, e = er.quantize8(x.double())
    assert torch.equal(kept.values.cpu(), q) and torch.equal(kept.exponents.cpu(), e)
