"""Edges of the operators around the tail on the GPU: rows that no expert owns,
orders of summation, waits that expire."""

import subprocess
import sys
from pathlib import Path

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300.binding import LatentTailError, Status, latent_tail_check

import block_reference as br
import gpu_helpers as gh
from test_gpu_block import EPS, check_backward, gen, norm_case, randn, weights4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def cut(offsets, N):
    """Offsets as expert_matvec4 takes them: cut to [0, N], then their running maximum."""
    return torch.tensor(offsets).clamp(0, N).cummax(0).values


# --------------------------------------------------- rows that no expert owns
@pytest.mark.parametrize("E,M,C,G", [(3, 16, 64, 32),        # the smallest tiles
                                     (3, 7168, 256, 64),     # 64-row tiles
                                     (3, 40960, 64, 32)])    # 256-row tiles
@pytest.mark.parametrize("N,offsets", [
    (20, [3, 5, 9, 12]),               # a rank's slice of a larger array
    (20, [20, 20, 20, 20]), (20, [7, 7, 7, 7]),
    (40, [37, 37, 38, 40]),
    (6, [6, 4, 2, 0]), (9, [5, 1, 7, 3]),  # backwards
    (6, [0, 100, 3, 2 ** 31 - 1]), (6, [-5, -1, 2, 6]), (6, [-9, -8, -8, -2 ** 31]),
])
def test_matvec4_zeros_every_row_that_no_expert_owns(N, offsets, E, M, C, G):
    g = gen(N + M)
    packed, scales = weights4(E, M, C, G, g)
    x = randn(N, C, g=g)
    owned = cut(offsets, N)
    x[:int(owned[0])] = float("nan")  # not read into any result
    out = torch.full((N, M), float("nan"), dtype=torch.bfloat16, device="cuda")
    lt.expert_matvec4(x, packed, scales, torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                      out=out)
    latent_tail_check()
    ref, mag = br.matvec4(x, packed, scales, owned)
    br.assert_within(out, ref, br.bf16_bound(ref, (C + 2) * br.U32 * mag))
    assert (out[:int(owned[0])] == 0).all() and (out[int(owned[-1]):] == 0).all()


# ------------------------------------------------------ waits that run out
def timed_out(call):
    """Runs a self-test whose waits expire."""
    assert call() == Status.OK
    with pytest.raises(LatentTailError) as e:
        latent_tail_check()
    assert e.value.status == Status.TIMEOUT
    latent_tail_check()  # the error word was cleared


@pytest.mark.parametrize("N,E,M,C,G", [
    (1, 1, 7168, 2048, 128),  # two boxes per stage
    (1, 1, 256, 7168, 64),    # four
    (64, 64, 2048, 512, 32),  # one, 256-row tiles
    (24, 1, 7168, 1024, 64),  # sixteen rows per pass
])
def test_matvec4_keeps_what_did_not_arrive_out_of_the_result(lib, N, E, M, C, G):
    g = gen(N + M)
    packed, scales = weights4(E, M, C, G, g)
    x = randn(N, C, g=g)
    offsets = None
    if E > 1:
        offsets = torch.arange(E + 1, device="cuda").clamp(max=N).to(torch.int32)
    ref = lt.expert_matvec4(x, packed, scales, offsets)
    stream = torch.cuda.current_stream().cuda_stream
    for copied in (0, 1, 5):
        out = torch.full_like(ref, float("nan"))
        timed_out(lambda: lib.latent_tail_selftest_expert_matvec4_timeout(
            x.data_ptr(), packed.data_ptr(), scales.data_ptr(),
            0 if offsets is None else offsets.data_ptr(), out.data_ptr(), N, E, M, C, G, copied,
            2000, stream))
        came = ~torch.isnan(out)
        assert torch.equal(out[came], ref[came])
        assert not came.all() and (came.any() or copied == 0)
    assert torch.equal(lt.expert_matvec4(x, packed, scales, offsets), ref)
    latent_tail_check()


def ptr(t):
    return 0 if t is None else t.data_ptr()


def kinds(c):
    """Gate kind and residual type as the C entry points take them."""
    gate = c["gate"]
    kind = 0 if gate is None else 2 if gate.dim() == 1 else 1 if gate.shape[1] == 1 else 3
    return kind, int(c["residual"].dtype == torch.float32)


def arrived(got, want, before):
    """Which elements are the call's result; all others must be as they were."""
    came = got == want
    assert torch.equal(got[~came].nan_to_num(7.0), before[~came].nan_to_num(7.0))
    return came


@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("T,H,gate,residual", [
    (2000, 520, "none", "bf16"), (1000, 1024, "channel", "fp32"), (700, 7168, "token", "bf16"),
    (400, 8192, "full", "fp32"), (170, 9152, "channel", "bf16"), (160, 16384, "full", "fp32")])
def test_residual_norm_leaves_rows_that_did_not_arrive_untouched(lib, T, H, gate, residual, post,
                                                                 nxt):
    c = norm_case(T, H, gate, residual, seed=T + H, post=post, nxt=nxt)
    v, z = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    stream = torch.cuda.current_stream().cuda_stream
    for copied in (0, 2, 154):
        r = c["residual"].clone()  # in place
        z2 = None if z is None else torch.full_like(z, float("nan"))
        timed_out(lambda: lib.latent_tail_selftest_residual_norm_timeout(
            ptr(c["block"]), ptr(r), ptr(c["post"]), ptr(c["gate"]), ptr(c["nxt"]), ptr(r),
            ptr(z2), T, H, *kinds(c), 1.0, EPS, copied, 2000, stream))
        came = arrived(r, v, c["residual"])
        assert came[:copied].all() and not came[copied:].all(1).any()
        if z is not None:
            came = arrived(z2, z, torch.full_like(z, float("nan")))
            assert came[:copied].all() and not came[copied:].any()
    again = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS, gate=c["gate"])
    assert torch.equal(again[0], v)
    latent_tail_check()


@pytest.mark.parametrize("T,H,gate,residual", [
    (1000, 520, "token", "bf16"), (2000, 1024, "channel", "fp32"), (700, 7168, "full", "bf16"),
    (170, 9152, "token", "bf16"), (160, 16384, "full", "fp32")])
def test_residual_norm_backward_leaves_rows_that_did_not_arrive_untouched(lib, T, H, gate,
                                                                          residual):
    c = norm_case(T, H, gate, residual, seed=T + H)
    g = gen(T)
    dv, dz = randn(T, H, g=g, dtype=c["residual"].dtype), randn(T, H, g=g)
    want = lt.residual_norm_backward(dv, dz, c["block"], c["residual"], c["post"], c["nxt"], EPS,
                                     gate=c["gate"])
    ws = torch.empty(lt.residual_norm_backward_workspace_size(T, H), dtype=torch.uint8,
                     device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for copied in (0, 2, 60):
        got = [torch.full_like(w, float("nan")) for w in want]
        timed_out(lambda: lib.latent_tail_selftest_residual_norm_backward_timeout(
            ptr(dv), ptr(dz), ptr(c["block"]), ptr(c["residual"]), ptr(c["post"]), ptr(c["gate"]),
            ptr(c["nxt"]), ptr(got[0]), ptr(got[1]), ptr(got[2]), ptr(got[3]), ptr(got[4]), T, H,
            *kinds(c), 1.0, EPS, ptr(ws), ws.numel(), copied, 2000, stream))
        for name, a, b in zip(("block", "residual", "post", "gate"), got, want):
            if name == "post" or a.dim() == 1:
                assert torch.isfinite(a).all()  # sums over the rows that came
                continue
            came = arrived(a, b, torch.full_like(a, float("nan")))
            assert came[:copied].all() and not came[copied:].any(), name
    again = lt.residual_norm_backward(dv, dz, c["block"], c["residual"], c["post"], c["nxt"], EPS,
                                      gate=c["gate"])
    for a, b in zip(again, want):
        assert torch.equal(a, b)
    latent_tail_check()


def test_selftest_limits(lib):
    call = lib.latent_tail_selftest_expert_matvec4_timeout
    for copied, limit in ((-1, 2000), (0, 0), (0, 1000001)):
        assert call(*[0x10000000] * 5, 1, 1, 8, 32, 32, copied, limit, None) == Status.INVALID_ARG
    call = lib.latent_tail_selftest_residual_norm_timeout
    assert call(*[0x10000000] * 7, 1, 8, 0, 0, 1.0, EPS, -1, 2000, None) == Status.INVALID_ARG
    call = lib.latent_tail_selftest_residual_norm_backward_timeout
    assert call(*[0x10000000] * 12, 1, 8, 0, 0, 1.0, EPS, 0x10000000, 64, 0, 0,
                None) == Status.INVALID_ARG


# ----------------------------------------------------------- first calls
FIRST_CALLS = """
import torch
import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
bf16 = lambda *s: torch.ones(*s, dtype=torch.bfloat16, device="cuda")
x, h, w = bf16(300, 256), bf16(300, 1024), torch.ones(1024, device="cuda")
ids = (torch.arange(2400, device="cuda").reshape(300, 8) % 5).int()
packed = torch.full((5, 64, 128), 0x99, dtype=torch.uint8, device="cuda")
scales = bf16(5, 64, 8)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    d = lt.dispatch(x, ids, 5)
    e = lt.expert_matvec4(d.rows, packed, scales, d.offsets)
    c = lt.combine(e, d.position)
    r, n = lt.residual_norm(h, h, w, w, 1e-6)
    b = lt.residual_norm_backward(h, h, h, h, w, w, 1e-6)
graph.replay()
lt.latent_tail_check()
assert (c == 8 * 256).all() and (r == 2).all() and ((n - 1).abs() < 1e-2).all()
assert b[0].isfinite().all()
"""


def test_first_calls_can_be_captured():
    """A process whose first calls of the operators, with their set-up, are in a capture."""
    root = Path(__file__).resolve().parents[1]
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr


# -------------------------------------- widths whose ring had no room for its CTAs
@pytest.mark.parametrize("T,H,gate", [(2000, 1000, "none"), (2000, 856, "full"),
                                      (1000, 1000, "channel"), (913, 856, "full")])
def test_residual_norm_backward_with_six_ctas_per_sm(T, H, gate):
    check_backward(norm_case(T, H, gate, "fp32", seed=T + H), seed=H)


# ------------------------------------------------------ orders of summation
@pytest.mark.parametrize("N", [1, 8, 40, 64, 130])
def test_matvec4_of_several_experts_across_tile_choices(N):
    """With several experts the number of rows decides into how many column parts a sum is
    cut, and so its order: the same row may differ in its last bits between calls of other
    lengths, within the bound of any order. One call gives the same bits every time."""
    E, M, C, G = 64, 2048, 1056, 32
    g = gen(5)
    packed, scales = weights4(E, M, C, G, g)
    x = randn(130, C, g=g)[:N].contiguous()
    offsets = (torch.arange(E + 1, device="cuda") * 3).clamp(max=N).to(torch.int32)
    out = lt.expert_matvec4(x, packed, scales, offsets)
    ref, mag = br.matvec4(x, packed, scales, offsets)
    br.assert_within(out, ref, br.bf16_bound(ref, (C + 2) * br.U32 * mag))
    assert torch.equal(out, lt.expert_matvec4(x, packed, scales, offsets))


# ----------------------------------------------------------- other streams
def test_every_operator_on_another_stream():
    """The outputs that a call allocates belong to the stream it is given."""
    g = gen(3)
    T, K, E, L, H = 600, 4, 9, 264, 1448
    c = norm_case(T, H, "channel", "bf16", seed=4)
    packed, scales = weights4(E, 72, 256, 64, g)
    x, x4, ids = randn(T, L, g=g), randn(T, 256, g=g), torch.randint(
        -1, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    w, go = torch.rand(T, K, generator=g, device="cuda"), randn(T, L, g=g)

    def calls(**on):
        d = lt.dispatch(x, ids, E, **on)
        e = lt.expert_matvec4(lt.dispatch(x4, ids, E, **on).rows, packed, scales, d.offsets, **on)
        out = lt.combine(d.rows, d.position, w, **on)
        back = lt.combine_backward(go, d.rows, d.position, w, **on)
        norm = lt.residual_norm(c["block"], c["residual"], c["post"], c["nxt"], EPS,
                                gate=c["gate"], **on)
        grads = lt.residual_norm_backward(norm[0], norm[1], c["block"], norm[0], c["post"],
                                          c["nxt"], EPS, gate=c["gate"], **on)
        return [*d, e, out, *back, *norm, *grads]

    want = calls()
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        got = calls(stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    latent_tail_check()


def test_autograd_takes_gradients_at_any_offset():
    rows = randn(6, 8, g=gen(5)).requires_grad_(True)
    position = torch.arange(6, dtype=torch.int32, device="cuda").reshape(3, 2)
    joined = torch.cat([rows.new_zeros(3), lta.combine_rows(rows, position).reshape(-1)])
    (joined * joined.detach()).float().sum().backward()
    out = rows.detach().float().reshape(3, 2, 8).sum(1).to(torch.bfloat16)
    assert torch.equal(rows.grad, out.repeat_interleave(2, 0))
