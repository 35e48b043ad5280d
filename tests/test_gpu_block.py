"""The operators around the tail on the GPU against their 64-bit forms: expert
dispatch, combine and its gradient, 4-bit expert products, fused residual norms
and their gradient. Bounds: see block_reference."""

import math

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300.binding import LatentTailError, Status, latent_tail_check

import block_reference as br
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def choices(T, K, E, seed, drop=0.0, skew=1.0):
    g = gen(seed)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits += skew * torch.randn(E, generator=g, device="cuda")
    ids = logits.topk(min(K, E), dim=1).indices.to(torch.int32)
    if K > E:
        ids = torch.randint(0, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        ids[torch.rand(T, K, generator=g, device="cuda") < drop] = -1
    return ids.contiguous()


def randn(*shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# --------------------------------------------------------------- dispatch
DISPATCH = [
    (1, 1, 1, 8, 0.0), (1, 8, 256, 2048, 0.0), (3, 5, 7, 72, 0.4), (16, 8, 256, 2048, 0.0),
    (5, 64, 4, 64, 0.3), (255, 8, 60, 136, 0.1), (256, 8, 256, 2048, 0.0), (257, 8, 256, 264, 0.0),
    (2048, 1, 1024, 16, 0.5), (2049, 1, 1024, 16, 0.5), (1013, 6, 60, 1448, 0.2),
    (4096, 8, 256, 2056, 0.0), (700, 3, 1, 4096, 0.0), (5000, 4, 513, 8, 0.9),
    (40, 2, 16, 16384, 0.1), (3001, 7, 1023, 16, 0.05),
]


@pytest.mark.parametrize("T,K,E,L,drop", DISPATCH)
def test_dispatch(T, K, E, L, drop):
    ids = choices(T, K, E, seed=T * 31 + K, drop=drop)
    x = randn(T, L, g=gen(T + L))
    rows = torch.full((T * K, L), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = lt.dispatch(x, ids, E, rows=rows)
    order, position, offsets = br.dispatch(ids, E)
    assert torch.equal(got.offsets.cpu(), offsets)
    assert torch.equal(got.order.cpu(), order)
    assert torch.equal(got.position.cpu(), position)
    want = x.cpu()[(order // K).long()]
    want[int(offsets[-1]):] = 0
    assert torch.equal(got.rows.cpu().view(torch.int16), want.view(torch.int16))
    alone = lt.dispatch(None, ids, E)
    assert alone.rows is None
    for a, b in zip(alone[1:], got[1:]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,K", [(9, 4), (3000, 4)])
def test_dispatch_of_ids_out_of_range(T, K):
    """Anything outside [0, E) is a choice without an expert."""
    E = 12
    ids = choices(T, K, E, seed=2)
    ids[::2, 0] = E
    ids[1::3, 1] = 2 ** 31 - 1
    ids[2::5, 2] = -2 ** 31
    got = lt.dispatch(randn(T, 64, g=gen(3)), ids, E)
    order, position, offsets = br.dispatch(ids, E)
    assert torch.equal(got.order.cpu(), order)
    assert torch.equal(got.position.cpu(), position)
    assert torch.equal(got.offsets.cpu(), offsets)


@pytest.mark.parametrize("T,K", [(7, 3), (4000, 2)])
@pytest.mark.parametrize("fill", [-1, 0, 5])
def test_dispatch_of_one_key(T, K, fill):
    """Nothing routed, or every choice on one expert."""
    ids = torch.full((T, K), fill, dtype=torch.int32, device="cuda")
    x = randn(T, 80, g=gen(4))
    got = lt.dispatch(x, ids, 6)
    order, position, offsets = br.dispatch(ids, 6)
    assert torch.equal(got.order.cpu(), order) and torch.equal(got.position.cpu(), position)
    assert torch.equal(got.offsets.cpu(), offsets)
    back = lt.combine(got.rows, got.position)
    assert torch.equal(back, (x.float() * K).to(torch.bfloat16) if fill >= 0
                       else torch.zeros_like(x))


def test_dispatch_rows_past_32_bit_element_offsets():
    T, K, E, L = (1 << 17) + 3, 8, 64, 2056
    assert T * K * L > 2 ** 31
    ids = choices(T, K, E, seed=5)
    x = randn(T, L, g=gen(6))
    got = lt.dispatch(x, ids, E)
    for a in range(0, T * K, 200_001):
        r = torch.arange(a, min(T * K, a + 5), device="cuda")
        assert torch.equal(got.rows[r], x[(got.order[r] // K).long()])
    assert torch.equal(got.rows[-3:], x[(got.order[-3:] // K).long()])
    w = torch.full((T, K), 0.125, device="cuda")
    back = lt.combine(got.rows, got.position, w)
    assert torch.equal(back, x)  # eighths of one row, summed exactly
    grad_rows, gw = lt.combine_backward(x, got.rows, got.position, w)
    assert torch.equal(grad_rows[-1], (x[int(got.order[-1]) // K].float() / 8).to(torch.bfloat16))
    want = (x[-2:].double() ** 2).sum(1, keepdim=True).expand(2, K)
    br.assert_within(gw[-2:], want, br.CHAIN * br.U32 * want)


def test_dispatch_on_another_stream_and_in_a_graph():
    T, K, E, L = 1000, 6, 40, 264
    ids, x = choices(T, K, E, seed=8), randn(T, L, g=gen(9))
    want = lt.dispatch(x, ids, E)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lt.dispatch(x, ids, E, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    w = torch.rand(T, K, generator=gen(10), device="cuda")
    ws = torch.empty(lt.dispatch_workspace_size(T, K, E), dtype=torch.uint8, device="cuda")
    bufs = [torch.empty_like(v) for v in want]
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = lt.dispatch(x, ids, E, *bufs, workspace=ws)
        lt.combine(d.rows, d.position, w, out=out)
    for seed in (11, 12):
        ids.copy_(choices(T, K, E, seed=seed, drop=0.2))
        graph.replay()
        torch.cuda.synchronize()
        ref = lt.dispatch(x, ids, E)
        for a, b in zip(bufs, ref):
            assert torch.equal(a, b)
        assert torch.equal(out, lt.combine(ref.rows, ref.position, w))


# ---------------------------------------------------------------- combine
COMBINE = [(1, 1, 1, 8, 0.0), (1, 8, 256, 2048, 0.0), (3, 5, 7, 72, 0.4), (16, 8, 256, 2048, 0.0),
           (5, 64, 64, 264, 0.3), (1013, 6, 60, 1448, 0.2), (333, 9, 60, 136, 0.1),
           (20, 17, 64, 16384, 0.2), (65, 3, 16, 520, 0.5), (130, 10, 20, 1024, 0.7)]


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,K,E,L,drop", COMBINE)
def test_combine_and_gradient(T, K, E, L, drop, weighted):
    g = gen(T * 7 + L)
    d = lt.dispatch(None, choices(T, K, E, seed=T + K, drop=drop), E)
    rows = randn(T * K, L, g=g)
    w = torch.rand(T, K, generator=g, device="cuda") if weighted else None
    out = lt.combine(rows, d.position, w)
    ref, mag = br.combine(rows, d.position, w)
    br.assert_within(out, ref, br.bf16_bound(ref, (K + 2) * br.U32 * mag), "combine")

    go = randn(T, L, g=g)
    grad_rows = torch.full_like(rows, float("nan"))
    grad_rows, gw = lt.combine_backward(go, rows, d.position, w, grad_rows=grad_rows)
    rr, rw, wmag = br.combine_backward(go, rows, d.position, w)
    br.assert_within(grad_rows, rr, br.bf16_bound(rr, br.U32 * rr.abs()), "grad_rows")
    br.assert_within(gw, rw, br.CHAIN * br.U32 * wmag, "grad_weights")
    only, none = lt.combine_backward(go, None, d.position, w)
    assert none is None and torch.equal(only, grad_rows)


def test_combine_is_the_gradient_of_dispatch():
    """<dispatch(x), R> = <x, combine(R)> for unweighted sums, in 64 bits."""
    T, K, E, L = 77, 4, 9, 136
    g = gen(21)
    x, R = randn(T, L, g=g), randn(T * K, L, g=g)
    d = lt.dispatch(x, choices(T, K, E, seed=22, drop=0.3), E)
    left = (d.rows.double() * R.double()).sum()
    ref, mag = br.combine(R, d.position, None)
    right = (x.double() * ref).sum()
    assert abs(left - right) <= 1e-12 * (x.double().abs() * mag).sum()
    got = lt.combine(R, d.position)
    br.assert_within(got, ref, br.bf16_bound(ref, (K + 2) * br.U32 * mag))


def test_combine_gradient_against_differences():
    """Directional differences of the 64-bit sum against the kernel's gradients."""
    T, K, E, L = 40, 5, 8, 264
    g = gen(23)
    d = lt.dispatch(None, choices(T, K, E, seed=24, drop=0.2), E)
    rows, go = randn(T * K, L, g=g), randn(T, L, g=g)
    w = torch.rand(T, K, generator=g, device="cuda")
    grad_rows, gw = lt.combine_backward(go, rows, d.position, w)
    dr = torch.randn(T * K, L, generator=g, device="cuda", dtype=torch.float64)
    dw = torch.randn(T, K, generator=g, device="cuda", dtype=torch.float64)
    h = 2.0 ** -10

    def loss(s):
        out, _ = br.combine(rows.double() + s * h * dr, d.position, w.double() + s * h * dw)
        return (out * go.double()).sum()

    # the loss is quadratic along the line: central differences are exact up to rounding
    diff = (loss(1) - loss(-1)) / (2 * h)
    got = (grad_rows.double() * dr).sum() + (gw.double() * dw).sum()
    # each bf16 element is at most UBF off, and the errors enter with |direction|
    bound = br.UBF * (grad_rows.double().abs() * dr.abs()).sum() + 1e-3
    assert abs(diff - got) <= bound


def test_values_in_skipped_places_do_not_matter():
    """NaN and infinities in rows and weights of choices without an expert stay out;
    in routed places they reach exactly their own outputs."""
    T, K, E, L = 9, 4, 5, 72
    g = gen(25)
    ids = choices(T, K, E, seed=26)
    ids[0] = -1
    ids[1, 2] = E + 3
    d = lt.dispatch(None, ids, E)
    rows = randn(T * K, L, g=g)
    w = torch.rand(T, K, generator=g, device="cuda")
    go = randn(T, L, g=g)
    ref, mag = br.combine(rows, d.position, w)
    n = int(d.offsets[-1])
    rows[n:] = float("nan")
    w[0] = float("nan")
    w[1, 2] = float("inf")
    go[0] = float("inf")
    out = lt.combine(rows, d.position, w)
    br.assert_within(out, ref, br.bf16_bound(ref, (K + 2) * br.U32 * mag))
    assert (out[0] == 0).all()
    grad_rows, gw = lt.combine_backward(go, rows, d.position, w)
    assert (grad_rows[n:] == 0).all() and (gw[0] == 0).all() and gw[1, 2] == 0
    assert torch.isfinite(grad_rows).all() and torch.isfinite(gw).all()
    r = int(d.position[3, 1])
    rows[r, 5] = float("nan")
    w[4, 0] = float("inf")
    out2 = lt.combine(rows, d.position, w)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[3] = keep[4] = False
    assert torch.equal(out2[keep], out[keep])
    assert torch.isnan(out2[3]).sum() == 1 and not torch.isfinite(out2[4]).any()


def test_positions_out_of_range_are_skipped():
    T, K, L = 6, 3, 64
    g = gen(27)
    rows, go = randn(T * K, L, g=g), randn(T, L, g=g)
    position = torch.arange(T * K, dtype=torch.int32, device="cuda").reshape(T, K)
    position[0, 0] = T * K
    position[2, 1] = 2 ** 31 - 1
    position[4, 2] = -2 ** 31
    ref, mag = br.combine(rows, position, None)
    br.assert_within(lt.combine(rows, position), ref, br.bf16_bound(ref, 5 * br.U32 * mag))
    grad_rows = torch.full_like(rows, 7.0)
    _, gw = lt.combine_backward(go, rows, position, grad_rows=grad_rows)
    for t, k in ((0, 0), (2, 1), (4, 2)):
        assert gw[t, k] == 0 and (grad_rows[t * K + k] == 7.0).all()  # no choice named that row


# ---------------------------------------------------------------- matvec4
def weights4(E, M, C, G, g):
    packed = torch.randint(0, 256, (E, M, C // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(E, M, C // G, generator=g, device="cuda")) / math.sqrt(21 * C)).to(
        torch.bfloat16)
    return packed, scales


def check_matvec4(x, packed, scales, offsets, what=""):
    N, C = x.shape
    out = torch.full((N, packed.shape[1]), float("nan"), dtype=torch.bfloat16, device="cuda")
    lt.expert_matvec4(x, packed, scales, offsets, out=out)
    ref, mag = br.matvec4(x, packed, scales, offsets)
    br.assert_within(out, ref, br.bf16_bound(ref, (C + 2) * br.U32 * mag), what)
    return out


@pytest.mark.parametrize("N,M,C,G", [
    (1, 8, 32, 32), (1, 7168, 2048, 128), (2, 72, 128, 64), (3, 264, 96, 32), (7, 40, 320, 64),
    (8, 128, 512, 128), (9, 24, 2048, 32), (16, 1000, 256, 128), (17, 136, 160, 32),
    (24, 520, 1152, 128), (33, 48, 2048, 64), (64, 256, 384, 128), (100, 16, 16384, 128),
    (1, 64, 16384, 32), (200, 152, 224, 32)])
def test_matvec4_dense(N, M, C, G):
    g = gen(N + M + C)
    packed, scales = weights4(1, M, C, G, g)
    x = randn(N, C, g=g)
    out = check_matvec4(x, packed, scales, None)
    offsets = torch.tensor([0, N], dtype=torch.int32, device="cuda")
    assert torch.equal(lt.expert_matvec4(x, packed, scales, offsets), out)


@pytest.mark.parametrize("T,K,E,M,C,G,drop", [
    (1, 8, 256, 128, 256, 32, 0.0), (16, 8, 64, 264, 512, 64, 0.0), (5, 3, 9, 40, 2048, 128, 0.5),
    (64, 8, 16, 72, 384, 128, 0.1), (40, 2, 3, 200, 96, 32, 0.0), (300, 4, 5, 16, 64, 32, 0.2),
    (2, 2, 1024, 24, 32, 32, 0.0), (50, 6, 7, 8, 128, 64, 0.97)])
def test_matvec4_experts(T, K, E, M, C, G, drop):
    g = gen(T + M)
    d = lt.dispatch(randn(T, C, g=g), choices(T, K, E, seed=T + E, drop=drop), E)
    packed, scales = weights4(E, M, C, G, g)
    out = check_matvec4(d.rows, packed, scales, d.offsets)
    assert (out[int(d.offsets[-1]):] == 0).all()


def test_matvec4_without_any_routed_row():
    packed, scales = weights4(4, 16, 64, 32, gen(1))
    d = lt.dispatch(randn(5, 64, g=gen(2)), torch.full((5, 2), -1, dtype=torch.int32,
                                                       device="cuda"), 4)
    out = torch.full((10, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    assert (lt.expert_matvec4(d.rows, packed, scales, d.offsets, out=out) == 0).all()


def test_matvec4_does_not_depend_on_the_other_rows():
    """A row's result has the same bits alone and among others (each output is one
    sum in an order that only the width fixes)."""
    g = gen(31)
    packed, scales = weights4(1, 136, 1152, 128, g)
    x = randn(40, 1152, g=g)
    whole = lt.expert_matvec4(x, packed, scales)
    for r in (0, 7, 8, 31, 39):
        assert torch.equal(lt.expert_matvec4(x[r:r + 1].clone(), packed, scales)[0], whole[r])


def test_matvec4_infinities_and_nan_stay_in_their_row():
    g = gen(32)
    packed, scales = weights4(1, 64, 256, 64, g)
    packed[0, :, 20] = 0x99  # weight (9 - 8): no zero times infinity
    x = randn(5, 256, g=g)
    ref = lt.expert_matvec4(x, packed, scales)
    x[1, 3] = float("nan")
    x[3, 40] = float("inf")
    out = lt.expert_matvec4(x, packed, scales)
    assert torch.isnan(out[1]).all() and torch.isinf(out[3]).all()
    for r in (0, 2, 4):
        assert torch.equal(out[r], ref[r])


def test_matvec4_large_and_tiny_magnitudes():
    g = gen(33)
    packed, scales = weights4(1, 32, 128, 32, g)
    for s in (2.0 ** 100, 2.0 ** -100):
        x = (torch.randn(3, 128, generator=g, device="cuda") * s).to(torch.bfloat16)
        check_matvec4(x, packed, scales, None, f"scale {s}")


def test_matvec4_weights_past_32_bit_offsets():
    E, M, C, G = 260, 8192, 4096, 128
    assert E * M * C // 2 > 2 ** 32
    g = gen(34)
    packed, scales = weights4(E, M, C, G, g)
    ids = torch.tensor([[0, E - 1], [E - 1, 129]], dtype=torch.int32, device="cuda")
    d = lt.dispatch(randn(2, C, g=g), ids, E)
    check_matvec4(d.rows, packed, scales, d.offsets)


def test_matvec4_reads_no_expert_beyond_bad_offsets():
    """Offsets that run backwards or past the rows are cut to [0, N]."""
    packed, scales = weights4(3, 16, 64, 32, gen(35))
    x = randn(6, 64, g=gen(36))
    for bad in ([0, 100, 3, 2 ** 31 - 1], [-5, -1, 2, 6], [6, 4, 2, 0]):
        offsets = torch.tensor(bad, dtype=torch.int32, device="cuda")
        lt.expert_matvec4(x, packed, scales, offsets)
    latent_tail_check()


def test_quantize4_round_trip():
    g = gen(37)
    w = torch.randn(48, 256, generator=g, device="cuda")
    w[3, 32:64] = 0
    packed, scales = lt.quantize4(w, 32)
    back = br.unpack4(packed, scales)[0]
    # q is at most half a step off, and the rounded scale can cut the largest value
    # by 7 * UBF of a step
    step = scales[0].double().repeat_interleave(32, dim=1)
    assert ((back - w.double()).abs() <= (0.5 + 7 * br.UBF) * step).all()
    check_matvec4(randn(4, 256, g=g), packed, scales, None)


# ---------------------------------------------------------- residual norms
def norm_case(T, H, gate, residual, seed, post=True, nxt=True):
    g = gen(seed)
    rt = torch.float32 if residual == "fp32" else torch.bfloat16
    gates = {"none": lambda: None,
             "token": lambda: torch.randn(T, 1, generator=g, device="cuda"),
             "channel": lambda: torch.randn(H, generator=g, device="cuda"),
             "full": lambda: randn(T, H, g=g)}
    w = lambda: 1 + 0.1 * torch.randn(H, generator=g, device="cuda")  # noqa: E731
    return dict(block=randn(T, H, g=g, scale=2.0), residual=randn(T, H, g=g, dtype=rt, scale=3.0),
                post=w() if post else None, nxt=w() if nxt else None, gate=gates[gate]())


def wide(v):
    return None if v is None else v.double()


def check_norm(c, scale=0.5, eps=EPS):
    v, z = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], eps, gate=c["gate"],
                            residual_scale=scale)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    rv, rz = br.residual_norm(wide(c["block"]), wide(c["residual"]), wide(c["post"]),
                              wide(c["gate"]), wide(c["nxt"]), scale, eps)
    u = rv - scale * wide(c["residual"])
    e = br.CHAIN * br.U32 * (u.abs() + (scale * wide(c["residual"])).abs())
    br.assert_within(v, rv, br.bf16_bound(rv, e) if v.dtype == torch.bfloat16 else e, "v")
    if rz is None:
        assert z is None
        return
    # z = v r2 w: v's own error, and that of r2, relative
    r2w = (c["nxt"].double() / torch.sqrt((rv * rv).mean(-1, keepdim=True) + eps)).abs()
    rel = e.square().mean(-1, keepdim=True).sqrt() / torch.sqrt(
        (rv * rv).mean(-1, keepdim=True) + eps) + br.CHAIN * br.U32
    br.assert_within(z, rz, br.bf16_bound(rz, e * r2w + rel * rz.abs()), "z")


SHAPES = [(1, 8), (3, 64), (9, 256), (5, 264), (7, 520), (4, 1024), (3, 1032), (1, 7168),
          (33, 5128), (2, 8192), (3, 8200), (2, 16384)]


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_residual_norm(T, H, residual, gate):
    check_norm(norm_case(T, H, gate, residual, seed=T + H))


@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("T,H", [(5, 264), (3, 7168), (2, 8200)])
def test_residual_norm_without_one_of_the_norms(T, H, post, nxt):
    check_norm(norm_case(T, H, "channel", "bf16", seed=H, post=post, nxt=nxt), scale=1.0)


def test_residual_norm_many_rows():
    check_norm(norm_case(4099, 1448, "token", "bf16", seed=4))
    check_norm(norm_case(4099, 72, "full", "fp32", seed=5))


def test_residual_norm_zero_rows_and_tiny_values():
    c = norm_case(4, 520, "none", "fp32", seed=6)
    c["block"][0] = 0
    c["residual"][1] = 0
    c["block"][1] = 0
    c["block"][2] *= 2.0 ** -40
    check_norm(c, scale=1.0)


def test_residual_norm_nan_stays_in_its_row():
    c = norm_case(9, 264, "channel", "bf16", seed=7)
    a = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    c["block"][4, 3] = float("nan")
    b = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    for x, y in zip(a, b):
        assert torch.isnan(y[4]).all()
        keep = [r for r in range(9) if r != 4]
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("H", [264, 7168, 8200])
def test_residual_norm_in_place(H, residual):
    c = norm_case(6, H, "token", residual, seed=8)
    v, z = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"],
                            residual_scale=0.5)
    r = c["residual"]
    v2, z2 = lt.residual_norm(c["block"], r, c["post"], c["nxt"], EPS, gate=c["gate"],
                              residual_scale=0.5, residual_out=r)
    assert v2 is r and torch.equal(r, v) and torch.equal(z2, z)


def reference_gradient(c, stored, dv, dz, scale, eps):
    """Gradients in 64 bits by differentiating the forward form at the residual input
    that gives ``stored``; also the terms' magnitudes for the sums over tokens."""
    block, post, gate, nxt = (wide(c[k]) for k in ("block", "post", "gate", "nxt"))
    for v in (block, post, gate, nxt):
        if v is not None:
            v.requires_grad_(True)
    with torch.no_grad():
        added, _ = br.residual_norm(block, torch.zeros_like(block), post, gate, None, scale, eps)
        residual = (stored.double() - added) / scale
    residual.requires_grad_(True)
    v, z = br.residual_norm(block, residual, post, gate, nxt, scale, eps)
    total = 0
    if dv is not None:
        total = total + (v * dv.double()).sum()
    if z is not None:
        total = total + (z * dz.double()).sum()
    total.backward()
    return [None if t is None else t.grad for t in (block, residual, post, gate, nxt)]


def check_backward(c, seed, scale=0.5, eps=EPS, grad_v=True):
    g = gen(seed)
    T, H = c["block"].shape
    stored = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], eps, gate=c["gate"],
                              residual_scale=scale)[0]
    dv = randn(T, H, g=g, dtype=stored.dtype) if grad_v else None
    dz = randn(T, H, g=g) if c["nxt"] is not None else None
    got = lt.residual_norm_backward(dv, dz, c["block"], stored, c["post"], c["nxt"], eps,
                                    gate=c["gate"], residual_scale=scale)
    scale = float(torch.tensor(scale, dtype=torch.float32))
    want = reference_gradient(c, stored, dv, dz, scale, eps)
    one = lambda v: 1.0 if v is None else v.double().abs()  # noqa: E731
    # Magnitudes of the terms of each gradient: the part along d (bounded by |dv| plus
    # the norm's two terms) and the part that the second norm subtracts.
    yb, vb = c["block"].double(), stored.double()
    r1 = 1 / torch.sqrt((yb * yb).mean(-1, keepdim=True) + eps) if c["post"] is not None else 1.0
    d = torch.zeros_like(vb) if dv is None else dv.double().abs()
    vh = None
    if dz is not None:
        r2 = 1 / torch.sqrt((vb * vb).mean(-1, keepdim=True) + eps)
        vh = (vb * r2).abs()
        a = dz.double().abs() * one(c["nxt"])
        d = d + r2 * (a + vh * (a * vh).mean(-1, keepdim=True))
    yh = (yb * r1).abs()
    b = d * one(c["gate"]) * one(c["post"])
    dy = r1 * (b + yh * (b * yh).mean(-1, keepdim=True)) if c["post"] is not None else b
    e = br.CHAIN * br.U32
    names = ["grad_block", "grad_residual", "grad_post", "grad_gate", "grad_next"]
    mags = [dy, scale * d, (d * one(c["gate"]) * yh).sum(0), None,
            None if vh is None else (dz.double().abs() * vh).sum(0)]
    gm = d * (yh * one(c["post"]) if c["post"] is not None else yb.abs())
    if c["gate"] is not None:
        mags[3] = gm.sum(0) if c["gate"].dim() == 1 else (
            gm.sum(1, keepdim=True) if c["gate"].shape[1] == 1 else gm)
    for name, x, ref, mag in zip(names, got, want, mags):
        if ref is None:
            assert x is None, name
            continue
        err = (e + T * br.U32 if name in ("grad_post", "grad_gate", "grad_next") else e) * mag
        br.assert_within(x, ref, br.bf16_bound(ref, err) if x.dtype == torch.bfloat16 else err,
                         name)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_residual_norm_backward(T, H, residual, gate):
    check_backward(norm_case(T, H, gate, residual, seed=T + H), seed=T * H)


@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["none", "channel"])
@pytest.mark.parametrize("H", [264, 7168, 8200])
def test_residual_norm_backward_without_one_of_the_norms(H, gate, post, nxt):
    check_backward(norm_case(3, H, gate, "bf16", seed=H, post=post, nxt=nxt), seed=H, scale=1.0)


@pytest.mark.parametrize("T,H", [(2500, 264), (1300, 1448), (700, 8200), (3001, 72)])
def test_residual_norm_backward_many_rows(T, H):
    check_backward(norm_case(T, H, "channel", "bf16", seed=9), seed=10)


def test_residual_norm_backward_without_the_outer_gradient():
    check_backward(norm_case(5, 520, "token", "bf16", seed=11), seed=12, grad_v=False)


def test_residual_norm_gradient_against_differences():
    """Directional differences of the 64-bit forward form against the kernel's gradients."""
    T, H, scale, h = 6, 264, 0.5, 1e-4
    c = norm_case(T, H, "channel", "fp32", seed=13)
    g = gen(14)
    stored = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"],
                              residual_scale=scale)[0]
    dv, dz = randn(T, H, g=g, dtype=torch.float32), randn(T, H, g=g)
    got = lt.residual_norm_backward(dv, dz, c["block"], stored, c["post"], c["nxt"], EPS,
                                    gate=c["gate"], residual_scale=scale)
    at = [wide(c[k]) for k in ("block", "residual", "post", "gate", "nxt")]
    for i, name in enumerate(("block", "residual", "post", "gate", "nxt")):
        step = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)

        def loss(s):
            p = list(at)
            p[i] = p[i] + s * h * step
            v, z = br.residual_norm(*p, scale, EPS)
            return (v * dv.double()).sum() + (z * dz.double()).sum()

        diff = (loss(1) - loss(-1)) / (2 * h)
        want = (got[i].double() * step).sum()
        # bf16 gradients: UBF per element; the rest: FP32 rounding, and h^2 times the third
        # derivative of the norms (about 1 per unit of the direction's size)
        off = br.UBF if got[i].dtype == torch.bfloat16 else br.CHAIN * br.U32
        bound = off * (got[i].double().abs() * step.abs()).sum() + 1e-4 * step.norm()
        assert abs(diff - want) <= bound, name


def test_results_are_the_same_bits_from_run_to_run():
    c = norm_case(1000, 1448, "channel", "bf16", seed=15)
    g = gen(16)
    dv, dz = randn(1000, 1448, g=g), randn(1000, 1448, g=g)
    first = lt.residual_norm_backward(dv, dz, c["block"], c["residual"], c["post"], c["nxt"], EPS,
                                      gate=c["gate"])
    for _ in range(3):
        again = lt.residual_norm_backward(dv, dz, c["block"], c["residual"], c["post"], c["nxt"],
                                          EPS, gate=c["gate"])
        for a, b in zip(first, again):
            assert torch.equal(a, b)


# ------------------------------------------------------- edges and refusals
def test_no_tokens():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    offsets = torch.full((6,), 9, dtype=torch.int32, device="cuda")
    d = lt.dispatch(z(0, 64), z(0, 4, dt=torch.int32), 5, offsets=offsets)
    assert (offsets == 0).all() and d.rows.shape == (0, 64)
    assert lt.combine(d.rows, d.position).shape == (0, 64)
    assert lt.combine_backward(z(0, 64), d.rows, d.position)[1].shape == (0, 4)
    packed, scales = weights4(5, 16, 64, 32, gen(1))
    assert lt.expert_matvec4(d.rows, packed, scales, offsets).shape == (0, 16)
    w = torch.ones(64, device="cuda")
    assert lt.residual_norm(z(0, 64), z(0, 64), w, w, EPS)[1].shape == (0, 64)
    got = lt.residual_norm_backward(z(0, 64), z(0, 64), z(0, 64), z(0, 64), w, w, EPS, gate=w)
    for v in (got[2], got[3], got[4]):
        assert v.shape == (64,) and (v == 0).all()


def test_refusals():
    g = gen(41)
    x, ids = randn(4, 64, g=g), choices(4, 2, 8, seed=42)
    d = lt.dispatch(x, ids, 8)
    bad = [
        (TypeError, lambda: lt.dispatch(x, ids.long(), 8)),
        (TypeError, lambda: lt.dispatch(x.float(), ids, 8)),
        (ValueError, lambda: lt.dispatch(x.t(), ids, 8)),
        (ValueError, lambda: lt.dispatch(x[:3], ids, 8)),
        (ValueError, lambda: lt.dispatch(x.cpu(), ids.cpu(), 8)),
        (ValueError, lambda: lt.dispatch(x.cpu(), ids, 8)),
        (ValueError, lambda: lt.dispatch(x, ids, 8, rows=torch.empty_like(x))),
        (ValueError, lambda: lt.combine(d.rows[:, ::2], d.position)),
        (TypeError, lambda: lt.combine(d.rows, d.position, torch.ones(4, 2, device="cuda",
                                                                       dtype=torch.bfloat16))),
        (ValueError, lambda: lt.combine(d.rows, d.position, torch.ones(2, 4, device="cuda"))),
        (TypeError, lambda: lt.residual_norm(x, x.double(), None, None, EPS)),
        (ValueError, lambda: lt.residual_norm(x, x, torch.ones(32, device="cuda"), None, EPS)),
        (TypeError, lambda: lt.residual_norm(x, x, None, None, EPS, gate=0.5)),
        (TypeError, lambda: lt.residual_norm(x, x, None, None, EPS, gate=x[:, :1])),  # bf16 [T, 1]
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
    packed, scales = weights4(8, 16, 64, 32, g)
    refused = [
        (Status.INVALID_ARG, lambda: lt.dispatch(x, ids, 1025)),
        (Status.INVALID_ARG, lambda: lt.expert_matvec4(d.rows, packed, scales)),  # 8 experts
        (Status.INVALID_ARG, lambda: lt.expert_matvec4(  # groups of 16 columns
            d.rows, packed, torch.ones(8, 16, 4, device="cuda", dtype=torch.bfloat16), d.offsets)),
        (Status.INVALID_ARG, lambda: lt.combine(d.rows, d.position, out=d.rows[:4])),
        (Status.INVALID_ARG, lambda: lt.residual_norm(x, x.clone(), None, None, 0.0)),
        (Status.INVALID_ARG, lambda: lt.residual_norm(x, x.clone(), None, None, EPS,
                                                      residual_scale=float("nan"))),
        (Status.INVALID_ARG, lambda: lt.residual_norm(x, x.clone(), None, None, EPS,
                                                      residual_out=x)),
        (Status.ALIGNMENT, lambda: lt.residual_norm(
            x, x.clone(), torch.ones(65, device="cuda")[1:], None, EPS)),
        (Status.INVALID_ARG, lambda: lt.residual_norm_backward(None, None, x, x.clone(), None,
                                                               None, EPS)),
        (Status.WORKSPACE, lambda: lt.residual_norm_backward(
            x, None, x, x.clone(), None, None, EPS,
            workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]
    for status, call in refused:
        with pytest.raises(LatentTailError) as err:
            call()
        assert err.value.status == status
    latent_tail_check()


# ------------------------------------------------ every kernel choice and its edges
@pytest.mark.parametrize("N,M,C,G", [
    (3, 8192, 256, 32),     # 64-row tiles; a row of scales shorter than a scale piece
    (5, 6600, 96, 32),      # ... scales read outside the ring
    (40, 7168, 320, 64),    # sixteen rows per pass, two and a half passes
    (13, 13000, 1056, 32),  # sixteen per pass, a last tile of eight rows
    (9, 40000, 128, 128),   # more tiles of 64 rows than CTAs
    (2, 200, 2816, 128),    # the smallest tiles, steps without all of their boxes
    (1, 131072, 512, 64),   # 256-row tiles of one matrix
])
def test_matvec4_dense_tile_choices(N, M, C, G):
    g = gen(N + M + C)
    packed, scales = weights4(1, M, C, G, g)
    check_matvec4(randn(N, C, g=g), packed, scales, None)


@pytest.mark.parametrize("T,K,E,M,C,G,drop", [
    (64, 8, 64, 2048, 256, 32, 0.1), (64, 8, 64, 2056, 96, 32, 0.0), (90, 8, 64, 1992, 1152, 128, 0.3),
    (300, 8, 70, 2000, 288, 32, 0.0), (128, 8, 64, 2048, 640, 64, 0.0), (33, 1, 256, 1024, 2048, 32, 0.0),
    (700, 2, 128, 1000, 64, 32, 0.1)])
def test_matvec4_experts_tile_choices(T, K, E, M, C, G, drop):
    g = gen(T + M)
    d = lt.dispatch(randn(T, C, g=g), choices(T, K, E, seed=T + E, drop=drop, skew=0.5), E)
    packed, scales = weights4(E, M, C, G, g)
    out = check_matvec4(d.rows, packed, scales, d.offsets)
    assert (out[int(d.offsets[-1]):] == 0).all()


RING = [(700, 4104), (613, 7168), (1300, 5128), (650, 8192)]


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", RING)
def test_residual_norm_rows_through_the_ring(T, H, residual, gate):
    c = norm_case(T, H, gate, residual, seed=T + H)
    check_norm(c)
    v, z = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"],
                            residual_scale=0.5)
    r = c["residual"].clone()
    v2, z2 = lt.residual_norm(c["block"], r, c["post"], c["nxt"], EPS, gate=c["gate"],
                              residual_scale=0.5, residual_out=r)
    assert torch.equal(v2, v) and torch.equal(z2, z)


@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (False, False)])
def test_residual_norm_ring_without_one_of_the_norms(post, nxt):
    check_norm(norm_case(611, 4800, "full", "bf16", seed=3, post=post, nxt=nxt))


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(700, 7168), (331, 8192), (1000, 520), (900, 1024), (1500, 2304),
                                 (800, 3584), (2000, 512)])
def test_residual_norm_backward_ring_depths(T, H, residual, gate):
    check_backward(norm_case(T, H, gate, residual, seed=T + H), seed=T * H)


def test_norm_rows_do_not_depend_on_the_other_rows():
    """Rows of a call through the ring have the same bits in a call of another length
    (a call of fewer rows than SMs takes another kernel, whose sums have another order)."""
    c = norm_case(1300, 4104, "channel", "bf16", seed=17)
    args = lambda n: (c["block"][:n].contiguous(), c["residual"][:n].contiguous(),  # noqa: E731
                      c["post"], c["nxt"], EPS)
    a = lt.residual_norm(*args(1300), gate=c["gate"])
    b = lt.residual_norm(*args(701), gate=c["gate"])
    for x, y in zip(a, b):
        assert torch.equal(x[:701], y)


@pytest.mark.parametrize("T,K,E,L", [(260, 8, 300, 2048), (2100, 1, 9, 8), (1200, 8, 64, 1024),
                                     (5200, 8, 64, 1024), (3000, 8, 40, 264), (300, 7, 1024, 4096)])
def test_dispatch_in_two_and_three_kernels(T, K, E, L):
    ids = choices(T, K, E, seed=T, drop=0.15)
    x = randn(T, L, g=gen(T + L))
    rows = torch.full((T * K, L), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = lt.dispatch(x, ids, E, rows=rows)
    order, position, offsets = br.dispatch(ids, E)
    assert torch.equal(got.offsets.cpu(), offsets)
    assert torch.equal(got.order.cpu(), order)
    assert torch.equal(got.position.cpu(), position)
    want = x.cpu()[(order // K).long()]
    want[int(offsets[-1]):] = 0
    assert torch.equal(got.rows.cpu().view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("L", [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056])
def test_combine_gradient_group_sizes(L):
    """One width on each side of every thread-group size."""
    T, K, E = 67, 9, 12
    g = gen(L)
    d = lt.dispatch(None, choices(T, K, E, seed=L, drop=0.2), E)
    rows, go = randn(T * K, L, g=g), randn(T, L, g=g)
    w = torch.rand(T, K, generator=g, device="cuda")
    grad_rows, gw = lt.combine_backward(go, rows, d.position, w)
    rr, rw, wmag = br.combine_backward(go, rows, d.position, w)
    br.assert_within(grad_rows, rr, br.bf16_bound(rr, br.U32 * rr.abs()), "grad_rows")
    br.assert_within(gw, rw, br.CHAIN * br.U32 * wmag, "grad_weights")


@pytest.mark.parametrize("one_key", [True, False])
def test_dispatch_of_the_most_choices(one_key):
    """2^24 choices: chunks of more than 16-bit counts allow with one per SM."""
    T, K, E = 1 << 21, 8, 5
    if one_key:
        ids = torch.full((T, K), 3, dtype=torch.int32, device="cuda")
        ids[7, 2] = 0
        ids[-1, -1] = -1
    else:
        ids = torch.randint(-1, E, (T, K), generator=gen(1), device="cuda", dtype=torch.int32)
    d = lt.dispatch(None, ids, E)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    assert torch.equal(d.order.long(), order)
    bounds = torch.searchsorted(key[order], torch.arange(E + 1, device="cuda"))
    assert torch.equal(d.offsets.long(), bounds)
    at = torch.arange(T * K, device="cuda")
    want = torch.empty_like(at)
    want[order] = torch.where(at < bounds[-1], at, -1 - at)
    assert torch.equal(d.position.reshape(-1).long(), want)


@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", ["token", "full"])
@pytest.mark.parametrize("T,H", [(5, 264), (9, 488), (7, 7168), (3, 8200), (700, 1448)])
def test_residual_norm_backward_gates_without_one_of_the_norms(T, H, gate, post, nxt):
    check_backward(norm_case(T, H, gate, "fp32", seed=H, post=post, nxt=nxt), seed=H)
    check_backward(norm_case(T, H, gate, "bf16", seed=H, post=post, nxt=nxt), seed=H + 1,
                   grad_v=not nxt)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(80, 8200), (160, 9152), (301, 12296), (153, 16384)])
def test_wide_rows_shared_by_two_ctas(T, H, residual, gate):
    c = norm_case(T, H, gate, residual, seed=T + H)
    check_norm(c)
    check_backward(c, seed=T * H)
    r = c["residual"].clone()
    v, z = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    v2, z2 = lt.residual_norm(c["block"], r, c["post"], c["nxt"], EPS, gate=c["gate"],
                              residual_out=r)
    assert torch.equal(v2, v) and torch.equal(z2, z)


@pytest.mark.parametrize("post,nxt", [(True, False), (False, True), (False, False)])
def test_wide_rows_without_one_of_the_norms(post, nxt):
    c = norm_case(170, 10008, "channel", "bf16", seed=3, post=post, nxt=nxt)
    check_norm(c, scale=1.0)
    check_backward(c, seed=4, scale=1.0)


@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("T,H", [(1030, 384), (1025, 512), (153, 520), (2500, 768), (305, 776),
                                 (915, 1024), (457, 1032), (921, 2304), (305, 2312), (640, 3584),
                                 (153, 3592), (611, 4096), (304, 5128), (305, 8192)])
def test_residual_norm_more_rows_than_the_gpu_works_on(T, H, residual, gate):
    check_norm(norm_case(T, H, gate, residual, seed=T + H))


@pytest.mark.parametrize("H", [512, 520, 1448, 3584, 7168, 9152, 12296, 16384])
def test_residual_norm_nan_and_in_place_with_many_rows(H):
    T = 333
    c = norm_case(T, H, "token", "bf16", seed=H)
    r = c["residual"].clone()
    v, z = lt.residual_norm(c["block"], r, c["post"], c["nxt"], EPS, gate=c["gate"])
    v2, z2 = lt.residual_norm(c["block"], r, c["post"], c["nxt"], EPS, gate=c["gate"],
                              residual_out=r)
    assert v2 is r and torch.equal(v2, v) and torch.equal(z2, z)
    c["block"][4, 3] = float("nan")
    c["residual"][T - 1, H - 1] = float("inf")
    v3, z3 = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    keep = [t for t in range(T) if t not in (4, T - 1)]
    assert torch.isnan(v3[4]).all() and torch.isnan(z3[4]).all()
    assert torch.equal(v3[keep], v[keep]) and torch.equal(z3[keep], z[keep])
    assert torch.equal(v3[T - 1, :-1], v[T - 1, :-1]) and torch.isinf(v3[T - 1, -1])


@pytest.mark.parametrize("T,H", [(1000, 520), (333, 1024), (2000, 2304), (777, 4096),
                                 (311, 4104), (700, 5128)])
def test_residual_norm_backward_sums_over_many_rows(T, H):
    for residual, gate in (("fp32", "full"), ("bf16", "channel")):
        check_backward(norm_case(T, H, gate, residual, seed=H), seed=T)


@pytest.mark.parametrize("T,K,L", [(3001, 1, 520), (400, 1, 4096), (701, 2, 1448), (16000, 2, 72),
                                   (300, 2, 16384), (999, 3, 264), (2000, 3, 1448),
                                   (640, 4, 4096), (1300, 4, 1032), (613, 5, 512)])
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_combine_and_gradient_of_few_choices(T, K, L, drop):
    g = gen(T + K)
    d = lt.dispatch(None, choices(T, K, 16, seed=T + L, drop=drop), 16)
    rows, go = randn(T * K, L, g=g), randn(T, L, g=g)
    w = torch.rand(T, K, generator=g, device="cuda")
    for weights in (w, None):
        out = lt.combine(rows, d.position, weights)
        ref, mag = br.combine(rows, d.position, weights)
        br.assert_within(out, ref, br.bf16_bound(ref, (K + 2) * br.U32 * mag), "combine")
    grad_rows = torch.full_like(rows, float("nan"))
    grad_rows, gw = lt.combine_backward(go, rows, d.position, w, grad_rows=grad_rows)
    rr, rw, wmag = br.combine_backward(go, rows, d.position, w)
    br.assert_within(grad_rows, rr, br.bf16_bound(rr, br.U32 * rr.abs()), "grad_rows")
    br.assert_within(gw, rw, br.CHAIN * br.U32 * wmag, "grad_weights")
    only, none = lt.combine_backward(go, None, d.position, w)
    assert none is None and torch.equal(only, grad_rows)
