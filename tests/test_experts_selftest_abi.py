"""Host-side checks of the self-tests of the experts' waits: what the call itself refuses,
and limits out of range (no GPU)."""

import pytest

from latent_moe_output_gb300 import binding
from latent_moe_output_gb300.binding import Status

# Fake, never-dereferenced addresses, 64 MiB apart.
A, B, C_, D, E_, F_ = (0x10000000 + 0x4000000 * i for i in range(6))
BAD, ALIGN, OK = Status.INVALID_ARG, Status.ALIGNMENT, Status.OK
LIMITS = [(dict(copied=-1), BAD), (dict(limit=0), BAD), (dict(limit=1000001), BAD)]


@pytest.fixture(scope="module")
def lib():
    from latent_moe_output_gb300 import build

    build.build()
    return binding.load_library()


@pytest.mark.parametrize("kwargs,expect", LIMITS + [
    (dict(N=-1), BAD), (dict(F=36), ALIGN), (dict(off=None), BAD), (dict(hidden=None), BAD),
    (dict(hidden=A), BAD), (dict(act=2), BAD), (dict(kind=1), BAD), (dict(kind=3), BAD),
    (dict(N=0), OK),
])
def test_gated(lib, kwargs, expect):
    p = dict(x=A, w=B, off=D, hidden=C_, saved=None, exps=None, N=40, E=4, F=32, C=64, act=0,
             kind=0, copied=0, limit=1000)
    p.update(kwargs)
    assert lib.latent_tail_selftest_expert_gated_timeout(*p.values(), None) == expect


@pytest.mark.parametrize("kwargs,expect", LIMITS + [
    (dict(N=-1), BAD), (dict(M=12), ALIGN), (dict(off=None), BAD), (dict(gx=None, gw=None), BAD),
    (dict(w=None), BAD), (dict(x=None), BAD), (dict(gx=A), BAD), (dict(gw=F_ + 4), ALIGN),
    (dict(N=0, gw=None), OK),
])
def test_matmul_backward(lib, kwargs, expect):
    p = dict(dy=A, x=B, w=C_, off=D, gx=E_, gw=F_, N=40, E=4, M=32, C=64, copied=0, limit=1000)
    p.update(kwargs)
    assert lib.latent_tail_selftest_expert_matmul_backward_timeout(*p.values(), None) == expect
