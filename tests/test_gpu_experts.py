"""The bf16 experts on the GPU against their 64-bit forms.

Places and sums are tested with integers, for which every product and every partial sum
is exact in FP32 (below 2^24), whatever the order: the result is the exact sum rounded
once. Roundings and the activation are tested with random values under derived bounds."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300.binding import LatentTailError, Status, latent_tail_check

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
    # sums over many rows of small matrices
    (5000, 1, 264, 200, None), (1023, 1, 72, 1000, None), (700, 1, 128, 32, None),
    # more tiles of one 32-row or 32-column chunk than two for each pair of CTAs
    (1300, 260, 264, 24, (5,) * 260),
    # columns of a weight gradient in narrower tiles
    (300, 1, 1000, 2568, None), (130, 3, 520, 1600, (50, 0, 80)),
]
IDS = [f"N{s[0]}E{s[1]}M{s[2]}C{s[3]}" for s in SHAPES]


@pytest.mark.parametrize("N,E,M,C,counts", SHAPES, ids=IDS)
def test_matmul_and_gradients_of_integers(N, E, M, C, counts):
    g = gen(N + M)
    offsets = None if counts is None else offs(*counts)
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
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


# ------------------------------------------------------------- random values
def tensor_core_error(mag, n):
    """FP32 error of a sum of n products of bf16 values (each product is exact): one rounding
    or truncation of 2^-23 per addition, of a magnitude of at most ``mag``."""
    return (n + 2) * 2 * br.U32 * mag


RANDOM = [(1, 1, 512, 1448, None), (24, 1, 256, 640, None), (70, 1, 128, 2056, None),
          (300, 4, 272, 712, (100, 0, 7, 180)), (12, 6, 64, 328, (1, 2, 3, 0, 2, 1))]


@pytest.mark.parametrize("N,E,M,C,counts", RANDOM)
def test_matmul_random(N, E, M, C, counts):
    g = gen(N * 7 + C)
    offsets = None if counts is None else offs(*counts)
    x, w = randn(N, C, g=g), randn(E, M, C, g=g, scale=C ** -0.5)
    want, mag = er.matmul(x, w, offsets)
    br.assert_within(lt.expert_matmul(x, w, offsets), want,
                     br.bf16_bound(want, tensor_core_error(mag, C)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("N,E,M,C,counts", RANDOM)
def test_gated_random(N, E, M, C, counts, act):
    """h = a(g) u: |a'| <= 1.13 for both activations, so an error dg of g and du of u moves h by
    at most 1.13 dg |u| + |a(g)| du + 1.13 dg du."""
    F = M // 2
    g = gen(N * 11 + C)
    offsets = None if counts is None else offs(*counts)
    x, w = randn(N, C, g=g), randn(E, 2 * F, C, g=g, scale=2 * C ** -0.5)
    pre, mag = er.matmul(x, w, offsets)
    gate, up = pre.chunk(2, dim=1)
    dg, du = tensor_core_error(mag, C).chunk(2, dim=1)
    want = er.act(gate, act) * up
    err = 1.13 * dg * (up.abs() + du) + er.act(gate, act).abs() * du + act_error(gate, act, want)
    saved = nan(N, 2, F)
    hidden = lt.expert_gated(x, w, offsets, activation=act, saved=saved)
    br.assert_within(hidden, want, br.bf16_bound(want, err))
    br.assert_within(saved, pre.unflatten(1, (2, F)),
                     br.bf16_bound(pre, tensor_core_error(mag, C)).unflatten(1, (2, F)))
    # In 8 bits: within half a unit of the value, and a unit is at most 1/63.5 of the largest.
    kept = lt.Checkpoint8.empty(N, 2, F)
    again = lt.expert_gated(x, w, offsets, activation=act, saved=kept)
    assert torch.equal(again, hidden)
    back = lt.dequantize8(kept).double()
    pre2 = pre.unflatten(1, (2, F))
    pad = torch.nn.functional.pad(pre2.abs(), (0, -F % 16)).unflatten(-1, (-1, 16)).amax(-1)
    top = pad.repeat_interleave(16, dim=-1)[..., :F]
    slack = tensor_core_error(mag, C).amax(1)[:, None, None]
    assert ((back - pre2).abs() <= (top + slack) / 127 + slack).all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "8bit"])
def test_gated_backward_random(act, save):
    """dg and du are rounded to bf16 (half a unit, 2^-8 of the value) before the products, and
    computed in FP32 within 2^-18 of their magnitudes: a' = s + g s' is a sum of terms of at
    most |s| + |g s'|, each within act_error's 2^-20 and the exponential's share, taken at
    |s| <= 30 here: 30 * 4 * 2^-24 < 2^-17 of itself at most."""
    N, E, F, C, counts = 300, 4, 136, 712, (100, 0, 7, 180)
    g = gen(5)
    offsets = offs(*counts)
    x, w, dh = randn(N, C, g=g), randn(E, 2 * F, C, g=g, scale=C ** -0.5), randn(N, F, g=g)
    kept = randn(N, 2, F, g=g, scale=1.5)
    saved = kept if save == "bf16" else lt.quantize8(kept)
    wide = kept.double() if save == "bf16" else er.dequantize8(*saved)
    wide.requires_grad_(True)
    mask = er.owned(offsets, N, E, "cuda")[:, None]
    h = er.act(wide[:, 0], act) * wide[:, 1]
    (pre,) = torch.autograd.grad(h, wide, dh.double())
    pre = pre.flatten(1) * mask
    gx, gw, hidden = lt.expert_gated_backward(dh, x, w, saved, offsets, activation=act)
    h = (h * mask).detach()
    br.assert_within(hidden, h, br.bf16_bound(h, act_error(wide[:, 0].detach(), act, h)))
    want = er.matmul_backward(pre, x, w, offsets)
    # magnitude of the terms of a' times the rest, for the FP32 error of dg
    gate, up = wide.detach().unbind(1)
    terms = torch.cat((dh.double().abs() * up.abs() * (1 + 1.2 * gate.abs()),
                       dh.double().abs() * gate.abs()), dim=1) * mask
    off = br.UBF * pre.abs() * (1 + br.UBF) + 2.0 ** -16 * terms
    mag = er.matmul_backward(off, x.abs(), w.abs(), offsets)
    sums = er.matmul_backward(pre.abs() + off, x.abs(), w.abs(), offsets)
    n = (2 * F, N)
    for i, got in enumerate((gx, gw)):
        br.assert_within(got, want[i],
                         br.bf16_bound(want[i], mag[i] + tensor_core_error(sums[i], n[i])))


def test_gated_gradient_against_differences():
    """(f(x + d) - f(x - d)) / 2 of f = sum(c h) in 64 bits along random directions."""
    N, E, F, C, counts = 40, 3, 72, 136, (15, 0, 20)
    g = gen(9)
    offsets = offs(*counts)
    x, w, c = randn(N, C, g=g), randn(E, 2 * F, C, g=g, scale=C ** -0.5), randn(N, F, g=g)
    saved = nan(N, 2, F)
    lt.expert_gated(x, w, offsets, saved=saved)
    gx, gw, _ = lt.expert_gated_backward(c, x, w, saved, offsets)

    def f(x, w):
        out = torch.zeros(N, 2 * F, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(er.bounds(offsets, N, E)):
            out[a:b] = x[a:b] @ w[e].t()
        gate, up = out.chunk(2, dim=1)
        return (er.act(gate, "silu") * up * c.double()).sum()

    for i, (t, grad) in enumerate(((x.double(), gx), (w.double(), gw))):
        d = torch.randn(t.shape, generator=g, device="cuda", dtype=torch.float64)
        step = 1e-4 * d
        args = lambda s: (t + s, w.double()) if i == 0 else (x.double(), t + s)  # noqa: E731
        want = (f(*args(step)) - f(*args(-step))) / 2e-4
        got = (grad.double() * d).sum()
        # Roundings to bf16 of g, u, dg, du and the gradient: five of 2^-8 each, of terms whose
        # sum along a random direction is about their norm; four norms is far in the tail.
        bound = 4 * 5 * br.UBF * (grad.double() * d).norm() + 1e-3 * want.abs()
        assert (got - want).abs() <= bound


# ---------------------------------------------------------- what must not spread
@pytest.mark.parametrize("N,E,M,C,counts,start", [
    (200, 3, 272, 200, (70, 33, 80), 0), (30, 3, 64, 72, (9, 5, 11), 2),
    (600, 3, 256, 128, (300, 100, 150), 13), (170, 3, 520, 1032, (50, 30, 70), 5)])
def test_nan_of_one_expert_stays_there(N, E, M, C, counts, start):
    """Rows and weights of expert 1, and rows that no expert owns, are NaN or infinite."""
    F = max(8, M // 16 * 8)
    g = gen(N)
    offsets = offs(*counts, start=start)
    (_, (a, b), _), mask = er.bounds(offsets, N, E), er.owned(offsets, N, E, "cuda")
    x, w, dy, up = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g), ints(E, 2 * F, C, g=g)
    good = mask.clone()
    good[a:b] = False
    clean = [t.clone() for t in (x, dy)]
    for t in (x, dy):
        t[~good] = float("nan")
        t[a] = float("inf")
    w[1], up[1] = float("nan"), float("inf")
    want = er.matmul(clean[0], w, offsets)[0]
    out = lt.expert_matmul(x, w, offsets, out=nan(N, M))
    same(out[good], want[good])
    assert torch.equal(out[~mask], torch.zeros_like(out[~mask]))
    gx, gw = lt.expert_matmul_backward(dy, x, w, offsets, grad_x=nan(N, C), grad_weights=nan(E, M, C))
    want = er.matmul_backward(clean[1], clean[0], w, offsets)
    same(gx[good], want[0][good])
    assert torch.equal(gx[~mask], torch.zeros_like(gx[~mask]))
    for e in (0, 2):
        same(gw[e], want[1][e])
    assert torch.isnan(gw[1]).all()
    saved = lt.Checkpoint8.empty(N, 2, F)
    hidden = lt.expert_gated(x, up, offsets, saved=saved)
    pre = er.matmul(clean[0], up, offsets)[0].unflatten(1, (2, F))
    q, e8 = er.quantize8(pre[good])
    assert torch.equal(saved.values[good], q) and torch.equal(saved.exponents[good], e8)
    assert torch.isnan(lt.dequantize8(saved)[a:b]).all()
    assert not saved.values[~mask].any() and not saved.exponents[~mask].any()
    assert not hidden[~mask].any() and torch.isfinite(hidden[good]).all()
    # kept projections of rows that no expert owns are not read
    kept = lt.dequantize8(saved)
    kept[a:b] = 0
    kept[~mask] = float("nan")
    gx, gw, h = lt.expert_gated_backward(clean[1][:, :F].contiguous() if M >= F else None, clean[0],
                                         up, kept, offsets)
    assert not gx[~mask].any() and not h[~mask].any()
    assert torch.isfinite(gx[good]).all() and torch.isfinite(gw[0]).all()


@pytest.mark.parametrize("raw,N", [
    ((5, 3, 9, 9), 12), ((-4, 2, 2 ** 30, 7), 12), ((40, 50, 60, 70), 12), ((9, 8, 7, 6), 12),
    ((0, 0, 0, 0), 100), ((0, 2 ** 31 - 1, -2 ** 31, 100), 300)])
def test_offsets_that_run_backwards_or_out_of_range(raw, N):
    offsets = torch.tensor(raw, dtype=torch.int32, device="cuda")
    E, M, C = 3, 72, 136
    g = gen(N)
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
    same(lt.expert_matmul(x, w, offsets, out=nan(N, M)), er.matmul(x, w, offsets)[0])
    gx, gw = lt.expert_matmul_backward(dy, x, w, offsets)
    want = er.matmul_backward(dy, x, w, offsets)
    same(gx, want[0])
    same(gw, want[1])
    saved = lt.Checkpoint8.empty(N, 2, 40)
    up = ints(E, 80, C, g=g)
    lt.expert_gated(x, up, offsets, saved=saved)
    same(lt.dequantize8(saved), er.dequantize8(*er.quantize8(
        er.matmul(x, up, offsets)[0].unflatten(1, (2, 40)))))
    latent_tail_check()


def test_one_row_and_many_experts():
    """1024 experts, most without rows, in every form."""
    E, M, C = 1024, 16, 24
    g = gen(1)
    counts = [0] * E
    for e, n in ((0, 1), (17, 40), (511, 300), (1000, 3), (1023, 2)):
        counts[e] = n
    offsets = offs(*counts)
    N = sum(counts) + 5
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
    same(lt.expert_matmul(x, w, offsets), er.matmul(x, w, offsets)[0])
    gx, gw = lt.expert_matmul_backward(dy, x, w, offsets, grad_weights=nan(E, M, C))
    want = er.matmul_backward(dy, x, w, offsets)
    same(gx, want[0])
    same(gw, want[1])
    for save in ("bf16", "8bit"):
        saved = nan(N, 2, 8) if save == "bf16" else lt.Checkpoint8.empty(N, 2, 8)
        lt.expert_gated(x, w, offsets, saved=saved)
        got = saved if save == "bf16" else lt.dequantize8(saved)
        pre = er.matmul(x, w, offsets)[0].unflatten(1, (2, 8))
        same(got, pre if save == "bf16" else er.dequantize8(*er.quantize8(pre)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gates_far_out(act):
    """Gates up to FP32's and bf16's limits: products and gradients as in 64 bits, where those
    are not near FP32's own."""
    values = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.0, -88.0, 104.0, -104.0, 1e4, -1e4, 1e30,
              -1e30, 3e38, -3e38]
    N, F, C = len(values), 8, 8
    kept = torch.ones(N, 2, F, dtype=BF16, device="cuda")
    kept[:, 0] = torch.tensor(values, device="cuda").to(BF16)[:, None]
    kept[:, 1] = 0.5
    dh = torch.full((N, F), 0.25, dtype=BF16, device="cuda")
    w = torch.zeros(1, 2 * F, C, dtype=BF16, device="cuda")
    w[0, :F] = torch.eye(F)
    gx, _, h = lt.expert_gated_backward(dh, None, w, kept, activation=act)
    wide = kept.double().requires_grad_(True)
    want = er.act(wide[:, 0], act) * wide[:, 1]
    (pre,) = torch.autograd.grad(want, wide, dh.double())
    want = want.detach()
    br.assert_within(h, want, br.bf16_bound(want, act_error(kept[:, 0].double(), act, want)))
    # s + g s': the second term is below 2^-24 of the first from |g| = 104 on, and the
    # reference's own is lost there (0 times infinity)
    d = torch.nan_to_num(pre[:, 0], nan=0.0)
    d = torch.where(kept[:, 0].double() >= 104, torch.full_like(d, 0.125), d)
    d = torch.where(kept[:, 0].double() <= -104, torch.zeros_like(d), d)
    br.assert_within(gx, d, 2 * br.UBF * d.abs() + 1e-6)
    nans = kept.clone()
    nans[3, 0, 2], nans[5, 1, 4], nans[7, 0, 1] = float("nan"), float("nan"), float("-inf")
    _, _, h = lt.expert_gated_backward(None, None, None, nans, activation=act)
    where = torch.zeros(N, F, dtype=torch.bool, device="cuda")
    where[3, 2] = where[5, 4] = where[7, 1] = True
    assert torch.equal(torch.isnan(h), where)


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("shape", [(1, 8), (1, 16), (3, 24), (16, 7168), (777, 5128), (5, 2, 40),
                                   (2, 3, 4, 8), (1, 65536), (1000, 16)])
def test_quantize8(shape):
    g = gen(shape[0])
    x = randn(*shape, g=g) * torch.exp(8 * torch.randn(shape[:-1] + (1,), generator=g,
                                                       device="cuda")).to(BF16)
    flat = x.view(-1, shape[-1])
    if flat.shape[0] > 2:
        flat[0] = 0
        flat[1, 0], flat[2, -1] = float("inf"), float("nan")
    want = er.quantize8(x.double())
    kept = lt.quantize8(x)
    assert torch.equal(kept.values, want[0]) and torch.equal(kept.exponents, want[1])
    back = er.dequantize8(*want)
    same(lt.dequantize8(kept), back)
    out = lt.Checkpoint8.empty(*shape)
    assert lt.quantize8(x, out) is out
    assert torch.equal(out.values, kept.values) and torch.equal(out.exponents, kept.exponents)


def test_quantize8_of_every_exponent():
    """Largest magnitudes just below, at and above 127.5 units, for every exponent of bf16."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    top = bits.to(torch.int16).view(BF16).cuda()
    x = torch.zeros(len(top), 16, dtype=BF16, device="cuda")
    x[:, 5] = -top
    x[:, 9] = top / 3
    x[:, 15] = top / 127
    want = er.quantize8(x.double())
    kept = lt.quantize8(x)
    assert torch.equal(kept.exponents, want[1]) and torch.equal(kept.values, want[0])
    same(lt.dequantize8(kept), er.dequantize8(*want))


def test_dequantize8_of_any_bytes():
    """Every value with every exponent, those that quantize8 does not write too."""
    values = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).cuda().repeat(256, 1)
    exponents = torch.arange(256, device="cuda").to(torch.uint8)[:, None].repeat(1, 16).contiguous()
    same(lt.dequantize8(lt.Checkpoint8(values, exponents)), er.dequantize8(values, exponents))


def test_more_elements_than_an_int_counts():
    T, C = 40008, 65536  # 2.6e9
    x = torch.empty(T, C, dtype=BF16, device="cuda").normal_(generator=gen(4))
    kept = lt.quantize8(x)
    back = lt.dequantize8(kept)
    for a in (0, 20000, T - 8):
        q, e = er.quantize8(x[a:a + 8].double())
        assert torch.equal(kept.values[a:a + 8], q) and torch.equal(kept.exponents[a:a + 8], e)
        same(back[a:a + 8], er.dequantize8(q, e))
    del kept, back
    # rows of a product past 2^31 elements in and out
    w = ints(1, 65536, 8, g=gen(5))
    narrow = ints(T, 8, g=gen(6))
    out = lt.expert_matmul(narrow, w)
    for a in (0, T - 300):
        same(out[a:a + 300], er.matmul(narrow[a:a + 300], w, None)[0])


# ------------------------------------------------------------ streams, graphs
def step(t, buffers):
    """The operators together: a training step's forward and backward pass."""
    x, up, down, dy, offsets = t
    lt.expert_gated(x, up, offsets, hidden=buffers["h"], saved=buffers["saved"])
    lt.expert_matmul(buffers["h"], down, offsets, out=buffers["y"])
    lt.expert_matmul_backward(dy, None, down, offsets, grad_x=buffers["dh"])
    lt.expert_gated_backward(buffers["dh"], x, up, buffers["saved"], offsets,
                             grad_x=buffers["dx"], grad_weights=buffers["dup"],
                             hidden=buffers["h2"], workspace=buffers["ws"])
    lt.expert_matmul_backward(dy, buffers["h2"], None, offsets, grad_weights=buffers["ddown"])


def step_state(seed, N=300, E=4, F=72, C=136, M=200):
    g = gen(seed)
    t = (randn(N, C, g=g), randn(E, 2 * F, C, g=g, scale=C ** -0.5),
         randn(E, M, F, g=g, scale=F ** -0.5), randn(N, M, g=g), offs(100, 0, 7, 180))
    b = dict(h=nan(N, F), saved=lt.Checkpoint8.empty(N, 2, F), y=nan(N, M), dh=nan(N, F),
             dx=nan(N, C), dup=nan(E, 2 * F, C), h2=nan(N, F), ddown=nan(E, M, F),
             ws=torch.empty(lt.expert_gated_backward_workspace_size(N, F), dtype=torch.uint8,
                            device="cuda"))
    return t, b


def results(b):
    return [t.clone() for k, v in sorted(b.items()) if k != "ws"
            for t in (v if isinstance(v, tuple) else (v,))]


def test_step_on_another_stream_and_in_a_graph():
    t, b = step_state(1)
    step(t, b)
    torch.cuda.synchronize()
    want = results(b)
    for _ in range(3):  # the same bits from call to call
        step(t, b)
    assert all(torch.equal(a, c) for a, c in zip(results(b), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, b2 = step_state(1)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(t, b2)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(results(b2), want))
    graph = torch.cuda.CUDAGraph()
    _, b3 = step_state(1)
    with torch.cuda.graph(graph):
        step(t, b3)
    t2, b4 = step_state(2)
    step(t2, b4)
    want2 = results(b4)
    for src, expected in ((t, want), (t2, want2), (t, want)):
        keep = [v.clone() for v in t]
        for dst, v in zip(t, src):
            dst.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(results(b3), expected))
        for dst, v in zip(t, keep):
            dst.copy_(v)
    latent_tail_check()


def test_calls_on_two_streams_at_once():
    states = [step_state(s, N=900, C=264, F=136) for s in (3, 4)]
    states = [((t[0], t[1], t[2], t[3], offs(200, 300, 0, 390)), b) for t, b in states]
    want = []
    for t, b in states:
        step(t, b)
        want.append(results(b))
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (t, b) in zip(streams, states):
            with torch.cuda.stream(s):
                step(t, b)
    torch.cuda.synchronize()
    for (t, b), w in zip(states, want):
        assert all(torch.equal(a, c) for a, c in zip(results(b), w))
    latent_tail_check()


def test_stream_argument():
    t, b = step_state(5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    x, up, down, dy, offsets = t
    torch.cuda.synchronize()
    got = [lt.expert_matmul(lt.expert_gated(x, up, offsets, stream=side), down, offsets,
                            stream=side)]
    kept = lt.quantize8(x, stream=side)
    got.append(lt.dequantize8(kept, stream=side.cuda_stream))
    got += lt.expert_matmul_backward(dy, got[0].new_zeros(300, 72), down, offsets, stream=side)
    side.synchronize()
    assert torch.equal(got[0], lt.expert_matmul(lt.expert_gated(x, up, offsets), down, offsets))
    assert torch.equal(got[1], lt.dequantize8(lt.quantize8(x)))


def test_no_rows():
    E, F, C, M = 3, 16, 24, 32
    x, up = nan(0, C), ints(E, 2 * F, C, g=gen(1))
    offsets = offs(0, 0, 0)
    assert lt.expert_gated(x, up, offsets).shape == (0, F)
    assert lt.expert_gated(x, up, offsets, saved=lt.Checkpoint8.empty(0, 2, F)).shape == (0, F)
    gx, gw, h = lt.expert_gated_backward(nan(0, F), x, up, nan(0, 2, F), offsets,
                                         grad_weights=nan(E, 2 * F, C))
    assert gx.shape == (0, C) and h.shape == (0, F) and not gw.any()
    down = ints(E, M, F, g=gen(2))
    assert lt.expert_matmul(nan(0, F), down, offsets).shape == (0, M)
    gx, gw = lt.expert_matmul_backward(nan(0, M), nan(0, F), down, offsets,
                                       grad_weights=nan(E, M, F))
    assert gx.shape == (0, F) and not gw.any()
    assert lt.dequantize8(lt.quantize8(nan(0, 40))).shape == (0, 40)


def test_refusals_on_the_gpu():
    x, w = nan(4, 64), nan(2, 32, 64)
    with pytest.raises(LatentTailError) as e:
        lt.expert_matmul(x, w)  # several experts without offsets
    assert e.value.status == Status.INVALID_ARG
    with pytest.raises(TypeError):
        lt.expert_matmul(x.float(), w[:1])
    with pytest.raises(ValueError):
        lt.expert_matmul(x.t(), w[:1])
    with pytest.raises(ValueError, match="contiguous"):
        lt.expert_matmul(nan(4, 128)[:, ::2], w[:1])
    with pytest.raises(ValueError, match="shape"):
        lt.expert_gated(x, w[:1], saved=nan(4, 2, 8))
    with pytest.raises(ValueError, match="device"):
        lt.expert_gated(x, w[:1].cpu())
    with pytest.raises(LatentTailError) as e:
        lt.expert_gated(nan(4 * 64 + 1)[1:].view(4, 64), w[:1])
    assert e.value.status == Status.ALIGNMENT
    with pytest.raises(LatentTailError) as e:
        lt.expert_gated_backward(nan(4, 16), x, w[:1], nan(4, 2, 16),
                                 workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == Status.WORKSPACE
    with pytest.raises(ValueError, match="without"):
        lt.expert_matmul_backward(nan(4, 32), x, None, grad_x=nan(4, 64))
    with pytest.raises(ValueError, match="activation"):
        lt.expert_gated(x, w[:1], activation="tanh")


# ------------------------------------------------------------- expired waits
@pytest.mark.parametrize("N,E,M,C,counts,copied", [
    (2000, 1, 2048, 256, None, 0), (2000, 1, 2048, 256, None, 40),
    (2000, 3, 1024, 256, (900, 0, 1000), 20),
    (100, 1, 512, 2048, None, 1)])   # several pairs per sum
def test_expired_waits_wind_down(lib, N, E, M, C, counts, copied):
    """Tiles that are never copied: the call ends, the status says so, and each element of out
    is the call's result or untouched. The next call is whole."""
    g = gen(N)
    offsets = None if counts is None else offs(*counts)
    x, w = ints(N, C, g=g), ints(E, M, C, g=g)
    want = lt.expert_matmul(x, w, offsets)
    latent_tail_check()
    out = torch.full((N, M), 16384.0, dtype=BF16, device="cuda")
    status = lib.latent_tail_selftest_expert_matmul_timeout(
        x.data_ptr(), w.data_ptr(), 0 if offsets is None else offsets.data_ptr(), out.data_ptr(),
        N, E, M, C, copied, 2000, torch.cuda.current_stream().cuda_stream)
    assert status == Status.OK
    with pytest.raises(LatentTailError) as e:
        latent_tail_check()
    assert e.value.status == Status.TIMEOUT
    untouched = out == 16384.0
    assert untouched.any()
    assert ((out == want) | untouched).all()
    if copied == 0:
        owned = er.owned(offsets, N, E, "cuda")
        assert untouched[owned].all()
    assert torch.equal(lt.expert_matmul(x, w, offsets), want)
    latent_tail_check()


def test_call_from_a_thread_without_a_context():
    """A thread whose first CUDA call this is: the driver has no context bound to it."""
    import threading

    g = gen(8)
    x, w = ints(100, 72, g=g), ints(1, 64, 72, g=g)
    out, want = nan(100, 64), lt.expert_matmul(x, w)
    lib, stream = gh.library(), torch.cuda.current_stream().cuda_stream
    args = (x.data_ptr(), w.data_ptr(), 0, out.data_ptr(), 100, 1, 64, 72, stream)
    torch.cuda.synchronize()
    got = []
    t = threading.Thread(target=lambda: got.append(lib.latent_tail_expert_matmul(*args)))
    t.start()
    t.join()
    assert got == [Status.OK]
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def random_shape(seed):
    """N, E, M, C and counts over the ranges where the kernels' choices change."""
    import random

    r = random.Random(seed)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** r.random()))  # noqa: E731
    N, M, C = log(1, 4000), 8 * log(1, 300), 8 * log(1, 300)
    if r.random() < 0.4:
        return N, 1, M, C, None, 0
    E = log(1, 300)
    M, C = min(M, 8 * (8000 // E + 1)), min(C, 1024)
    cuts = sorted(r.randint(0, N) for _ in range(E - 1))
    start, end = (r.randint(0, N // 8), N - r.randint(0, N // 8)) if r.random() < 0.5 else (0, N)
    cuts = [min(max(c, start), end) for c in cuts]
    edges = [start] + cuts + [end]
    return N, E, M, C, [b - a for a, b in zip(edges[:-1], edges[1:])], start


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes_of_integers(seed):
    N, E, M, C, counts, start = random_shape(seed)
    F = max(8, M // 16 * 8)
    g = gen(seed)
    offsets = None if counts is None else offs(*counts, start=start)
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
    same(lt.expert_matmul(x, w, offsets, out=nan(N, M)), er.matmul(x, w, offsets)[0], "out")
    got = lt.expert_matmul_backward(dy, x, w, offsets, grad_x=nan(N, C), grad_weights=nan(E, M, C))
    for a, b in zip(got, er.matmul_backward(dy, x, w, offsets)):
        same(a, b, "gradient")
    up = ints(E, 2 * F, C, g=g, most=1)
    pre = er.matmul(x, up, offsets)[0].unflatten(1, (2, F))
    saved = nan(N, 2, F) if seed % 2 else lt.Checkpoint8.empty(N, 2, F)
    hidden = lt.expert_gated(x, up, offsets, hidden=nan(N, F), saved=saved)
    if seed % 2:
        same(saved, pre, "saved")
    else:
        same(lt.dequantize8(saved), er.dequantize8(*er.quantize8(pre)), "saved")
    want = er.act(pre[:, 0], "silu") * pre[:, 1]
    br.assert_within(hidden, want, br.bf16_bound(want, act_error(pre[:, 0], "silu", want)))
    latent_tail_check()
