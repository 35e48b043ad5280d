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
