"""The bf16 experts on the GPU against their 64-bit forms.

Places and sums are tested with integers, for which every product and every partial sum
is exact in FP32 (below 2^24), whatever the order: the result is the exact sum rounded
once. Roundings and the activation are tested with random values under derived bounds."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300.binding import latent_tail_check

import block_reference as br
import experts_reference as er
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(*shape, g, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(BF16)


def randn(*shape, g, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


def nan(*shape):
    return torch.full(shape, float("nan"), dtype=BF16, device="cuda")


def offs(*counts, start=0):
    v = [start]
    for c in counts:
        v.append(v[-1] + c)
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def same(got, want64, what=""):
    """Bit for bit the exact value rounded to bf16 (zeros of either sign)."""
    want = want64.to(BF16)
    bad = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           got[bad][:4].tolist(), want[bad][:4].tolist())


def act_error(gate, act, value):
    """FP32 error of a(g) u: exponential, sum, reciprocal and two products are off by 2^-22
    each at most, 2^-20 in all; the exponential's argument by at most four roundings (the
    cubic of gelu has three), and the exponential by as much of itself as its argument
    is off. Where the sigmoid leaves FP32's normal numbers the product is below 1e-30."""
    s = er.act_argument(gate, act).abs()
    return (2.0 ** -20 + 4 * br.U32 * s.clamp(max=100)) * value.abs() + 1e-30


# N, E, M, C, offsets (None: one matrix for all rows)
SHAPES = [
    (1, 1, 8, 8, None), (1, 1, 256, 64, None), (2, 1, 264, 72, None), (15, 1, 128, 128, None),
    (16, 1, 1000, 136, None), (17, 1, 512, 64, None), (129, 1, 304, 200, None),
    (256, 1, 256, 512, None), (257, 1, 520, 1448, None), (1000, 1, 2048, 384, None),
    (40, 5, 64, 64, (8, 0, 17, 1, 14)), (700, 3, 136, 264, (300, 1, 399)),
    (300, 4, 712, 80, (0, 0, 290, 0)),                 # rows behind the last expert's
    (64, 3, 72, 96, (16, 16, 16)),                     # whole groups of 16
    (1030, 2, 256, 128, (513, 517)), (90, 9, 40, 40, (10,) * 9),
    (3, 300, 16, 16, (0,) * 200 + (1, 0, 1) + (0,) * 96 + (1,)),
    (2000, 7, 264, 328, (5, 700, 0, 3, 1000, 64, 100)),
    # sums shared by several pairs
    (33, 1, 512, 2048, None), (128, 1, 264, 1032, None), (200, 1, 1000, 1096, None),
    (60, 1, 4096, 512, None), (100, 4, 256, 1024, (10, 40, 0, 48)),
    # columns of a weight gradient in narrower tiles
    (300, 1, 1000, 2568, None), (130, 3, 520, 1600, (50, 0, 80)),
]
IDS = [f"N{s[0]}E{s[1]}M{s[2]}C{s[3]}" for s in SHAPES]


@pytest.mark.parametrize("N,E,M,C,counts", SHAPES, ids=IDS)
def test_matmul_and_gradients_of_integers(N, E, M, C, counts):
    g = gen(N + M)
    offsets = None if counts is None else offs(*counts)
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
    # More than twice the rows of a tile on either side of the arrays stay what they were.
    out, gx, gw = nan(N, M), nan(N, C), nan(E, M, C)
    lt.expert_matmul(x, w, offsets, out=out)
    latent_tail_check()
    same(out, er.matmul(x, w, offsets)[0], "out")
    lt.expert_matmul_backward(dy, x, w, offsets, grad_x=gx, grad_weights=gw)
    latent_tail_check()
    want = er.matmul_backward(dy, x, w, offsets)
    same(gx, want[0], "grad_x")
    same(gw, want[1], "grad_weights")


@pytest.mark.parametrize("N,E,M,C,counts", SHAPES, ids=IDS)
@pytest.mark.parametrize("save", ["none", "bf16", "8bit"])
def test_gated_of_integers(N, E, M, C, counts, save):
    """Kept projections exactly; products under the bound of one rounding (see ``act_error``)."""
    F = max(8, M // 16 * 8)
    g = gen(N + M + 1)
    offsets = None if counts is None else offs(*counts)
    x, w = ints(N, C, g=g, most=1), ints(E, 2 * F, C, g=g, most=2)
    saved = None
    if save == "bf16":
        saved = nan(N, 2, F)
    elif save == "8bit":
        saved = lt.Checkpoint8.empty(N, 2, F)
        saved.values.fill_(77)
        saved.exponents.fill_(200)
    pre, _ = er.matmul(x, w, offsets)
    gate, up = pre.chunk(2, dim=1)
    for act in ("silu", "gelu"):
        hidden = lt.expert_gated(x, w, offsets, activation=act, hidden=nan(N, F), saved=saved)
        latent_tail_check()
        want = er.act(gate, act) * up
        br.assert_within(hidden, want, br.bf16_bound(want, act_error(gate, act, want)), act)
        if save == "bf16":
            same(saved, pre.unflatten(1, (2, F)), "saved")
        elif save == "8bit":
            q, e = er.quantize8(pre.unflatten(1, (2, F)))
            assert torch.equal(saved.exponents, e)
            assert torch.equal(saved.values, q)


@pytest.mark.parametrize("N,E,M,C,counts", SHAPES, ids=IDS)
@pytest.mark.parametrize("save", ["bf16", "8bit"])
def test_gated_backward_of_integers(N, E, M, C, counts, save):
    """Gates of 64 (sigmoid 1 in FP32: a = 64, a' = 1) and -112 (sigmoid 0: a = a' = 0), ups
    and gradients small integers: dg and du are exact in bf16, and so are all sums."""
    F = max(8, M // 16 * 8)
    g = gen(N + M + 2)
    offsets = None if counts is None else offs(*counts)
    x, w, dh = ints(N, C, g=g), ints(E, 2 * F, C, g=g), ints(N, F, g=g, most=2)
    on = torch.randint(0, 2, (N, F), generator=g, device="cuda").bool()
    gate = torch.where(on, 64.0, -112.0).to(BF16)
    up = ints(N, F, g=g, most=4)
    kept = torch.stack((gate, up), dim=1).contiguous()
    saved = kept if save == "bf16" else lt.quantize8(kept)
    gx, gw, h = lt.expert_gated_backward(dh, x, w, saved, offsets, hidden=nan(N, F),
                                         grad_x=nan(N, C), grad_weights=nan(E, 2 * F, C))
    latent_tail_check()
    mask = er.owned(offsets, N, E, "cuda")[:, None]
    pre = torch.cat((dh.double() * up.double() * on, dh.double() * 64 * on), dim=1) * mask
    want = er.matmul_backward(pre, x, w, offsets)
    same(h, 64.0 * on * up.double() * mask, "hidden")
    same(gx, want[0], "grad_x")
    same(gw, want[1], "grad_weights")
