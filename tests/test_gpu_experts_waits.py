"""Waits of the experts' kernels that run out: the call ends soon, every element is the
call's result or untouched, and the next call is whole."""

import time

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300.binding import LatentTailError, Status, latent_tail_check

import experts_reference as er
import gpu_helpers as gh

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
MARK = 16384.0  # of an element that no call has written
ALL = 2 ** 31 - 1  # copied tiles: every one


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(*shape, g, most=3):
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(BF16)


def offs(*counts):
    v = [0]
    for c in counts:
        v.append(v[-1] + c)
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def marked(*shape):
    return torch.full(shape, MARK, dtype=BF16, device="cuda")


def ptr(t):
    return 0 if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


def ended_by(run):
    """Status that the device reports of a call, which ends well before a wait of a second
    would: copies on their way are waited for as long as they take, and no longer."""
    torch.cuda.synchronize()
    t0 = time.monotonic()
    assert run() == Status.OK
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 0.5
    try:
        latent_tail_check()
    except LatentTailError as e:
        return e.status
    return Status.OK


def whole_or_untouched(got, want):
    untouched = got == MARK
    assert ((got == want) | untouched).all()
    return untouched


# N, M, C, counts: one matrix, experts, several pairs per sum
PRODUCTS = [(2000, 2048, 1096, None), (2000, 1024, 256, (900, 0, 1000)), (100, 512, 2048, None),
            (200, 1000, 1096, None)]


@pytest.mark.parametrize("N,M,C,counts", PRODUCTS)
@pytest.mark.parametrize("copied", [1, 77, ALL])
def test_copies_on_their_way_when_a_wait_runs_out(lib, N, M, C, counts, copied):
    """Limits about as long as a copy takes: the CTAs of a pair give up with copies under way,
    and not after the same number of blocks."""
    g = gen(N + M)
    E = 1 if counts is None else len(counts)
    offsets = None if counts is None else offs(*counts)
    x, w = ints(N, C, g=g), ints(E, M, C, g=g)
    want = lt.expert_matmul(x, w, offsets)
    seen = set()
    for limit in (1, 2, 3, 5, 8, 20) * 4:
        out = marked(N, M)
        seen.add(ended_by(lambda: lib.latent_tail_selftest_expert_matmul_timeout(
            ptr(x), ptr(w), ptr(offsets), ptr(out), N, E, M, C, copied, limit, stream())))
        whole_or_untouched(out, want)
        assert torch.equal(lt.expert_matmul(x, w, offsets), want)
        latent_tail_check()
    assert copied != 1 or Status.TIMEOUT in seen  # (77 is every tile of some shapes)


# N, E, F, C, counts
GATED = [(2000, 1, 1024, 264, None), (1903, 3, 512, 520, (900, 0, 1000)),
         (100, 1, 256, 2048, None)]  # several pairs per sum


@pytest.mark.parametrize("N,E,F,C,counts", GATED)
@pytest.mark.parametrize("save", ["none", "bf16", "8bit"])
def test_gated(lib, N, E, F, C, counts, save):
    g = gen(N + F)
    offsets = None if counts is None else offs(*counts)
    x, w = ints(N, C, g=g, most=1), ints(E, 2 * F, C, g=g, most=2)

    def buffers():
        if save == "none":
            return ()
        if save == "bf16":
            return (marked(N, 2, F),)
        kept = lt.Checkpoint8.empty(N, 2, F)
        kept.values.fill_(-128)  # (which quantize8 does not write)
        kept.exponents.fill_(254)
        return tuple(kept)

    def saved_of(b):
        return None if not b else b[0] if len(b) == 1 else lt.Checkpoint8(*b)

    want_saved = buffers()
    want = lt.expert_gated(x, w, offsets, saved=saved_of(want_saved))
    latent_tail_check()
    for copied in (0, 1, 7, ALL):
        for limit in (1, 5, 20, 2000):
            hidden, kept = marked(N, F), buffers()
            status = ended_by(lambda: lib.latent_tail_selftest_expert_gated_timeout(
                ptr(x), ptr(w), ptr(offsets), ptr(hidden), ptr(kept[0] if kept else None),
                ptr(kept[1] if len(kept) == 2 else None), N, E, F, C, 0,
                ("none", "bf16", "8bit").index(save), copied, limit, stream()))
            untouched = whole_or_untouched(hidden, want)
            for a, b, m in zip(kept, want_saved, (MARK,) if save == "bf16" else (-128, 254)):
                assert ((a == b) | (a == m)).all()
            if copied <= 1:
                assert status == Status.TIMEOUT and untouched.any()
            if copied == 0:
                owned = er.owned(offsets, N, E, "cuda")
                assert untouched[owned].all() and not hidden[~owned].any()
            if status == Status.OK:
                assert not untouched.any()
            assert torch.equal(lt.expert_gated(x, w, offsets), want)
            latent_tail_check()


# N, E, M, C, counts: ends inside an MMA's 16 rows, whole groups of 16, experts without rows,
# sums over many rows that several pairs share
BACKWARD = [(1903, 3, 512, 520, (900, 0, 1003)), (1904, 2, 520, 256, (896, 1008)),
            (300, 9, 264, 1024, (10, 33, 0, 64, 1, 100, 50, 31, 11)), (5001, 1, 264, 200, None),
            (1000, 1, 1000, 264, None), (1023, 1, 72, 1000, None)]


@pytest.mark.parametrize("N,E,M,C,counts", BACKWARD)
def test_gradients_of_a_product(lib, N, E, M, C, counts):
    g = gen(N + M)
    offsets = None if counts is None else offs(*counts)
    x, w, dy = ints(N, C, g=g), ints(E, M, C, g=g), ints(N, M, g=g)
    want = lt.expert_matmul_backward(dy, x, w, offsets)
    latent_tail_check()
    empty = [e for e, (a, b) in enumerate(er.bounds(offsets, N, E)) if a == b]
    for copied in (0, 1, 5, ALL):
        for limit in (1, 5, 20, 2000):
            gx, gw = marked(N, C), marked(E, M, C)
            status = ended_by(lambda: lib.latent_tail_selftest_expert_matmul_backward_timeout(
                ptr(dy), ptr(x), ptr(w), ptr(offsets), ptr(gx), ptr(gw), N, E, M, C, copied, limit,
                stream()))
            left = [whole_or_untouched(a, b) for a, b in zip((gx, gw), want)]
            if copied == 0:
                owned = er.owned(offsets, N, E, "cuda")
                assert status == Status.TIMEOUT and left[0][owned].all()
                assert all(left[1][e].all() for e in range(E) if e not in empty)
            if status == Status.OK:
                assert not left[0].any() and not left[1].any()
            again = lt.expert_matmul_backward(dy, x, w, offsets)
            assert all(torch.equal(a, b) for a, b in zip(again, want))
            latent_tail_check()


def test_a_limit_is_of_one_wait_and_not_of_the_work_before_it(lib):
    """Tiles whose rows end inside an MMA's 16 come last here, 3 ms of healthy work after the
    first; a wait may take 1 ms."""
    counts, M, C = (16384, 8), 16384, 16384
    N, E = sum(counts), len(counts)
    g = gen(1)
    offsets = offs(*counts)
    x, dy = ints(N, C, g=g), ints(N, M, g=g)
    want = lt.expert_matmul_backward(dy, x, None, offsets)[1]
    got = marked(E, M, C)
    status = ended_by(lambda: lib.latent_tail_selftest_expert_matmul_backward_timeout(
        ptr(dy), ptr(x), 0, ptr(offsets), 0, ptr(got), N, E, M, C, ALL, 1000, stream()))
    assert status == Status.OK
    assert torch.equal(got, want)
