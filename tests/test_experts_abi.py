"""Host-side checks of the bf16 experts and of activations in 8 bits: bad arguments are
refused before any CUDA call, on a machine without a GPU too."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300 import binding
from latent_moe_output_gb300.binding import Status

import experts_reference as er

# Fake, never-dereferenced addresses, 64 MiB apart.
A, B, C_, D, E_, F_, G, H, I, WS = (0x10000000 + 0x4000000 * i for i in range(10))
BAD, ALIGN, OK = Status.INVALID_ARG, Status.ALIGNMENT, Status.OK


@pytest.fixture(scope="module")
def lib():
    from latent_moe_output_gb300 import build

    build.build()
    return binding.load_library()


SIZES = [
    (dict(N=-1), BAD), (dict(N=(1 << 24) + 1), BAD), (dict(E=0), BAD), (dict(E=1025), BAD),
    (dict(C=4), BAD), (dict(C=65544), BAD), (dict(C=60), ALIGN), (dict(off=None), BAD),
    (dict(off=D + 4), ALIGN), (dict(x=None), BAD), (dict(w=None), BAD), (dict(x=A + 8), ALIGN),
]


def gated(lib, x=A, w=B, off=D, hidden=C_, saved=None, exps=None, N=40, E=4, F=32, C=64, act=0,
          kind=0):
    return lib.latent_tail_expert_gated(x, w, off, hidden, saved, exps, N, E, F, C, act, kind, None)


@pytest.mark.parametrize("kwargs,expect", SIZES + [
    (dict(F=4), BAD), (dict(F=32776), BAD), (dict(F=36), ALIGN), (dict(hidden=None), BAD),
    (dict(act=2), BAD), (dict(act=-1), BAD), (dict(kind=3), BAD), (dict(kind=1), BAD),
    (dict(saved=E_), BAD), (dict(kind=2, saved=E_), BAD), (dict(kind=1, saved=E_, exps=F_), BAD),
    (dict(kind=1, saved=E_ + 8), ALIGN), (dict(kind=2, saved=E_, exps=F_ + 1), ALIGN),
    (dict(hidden=A + 64), BAD), (dict(hidden=B), BAD), (dict(kind=1, saved=C_ + 16), BAD),
    (dict(kind=2, saved=E_, exps=E_ + 64), BAD), (dict(hidden=D), BAD),
    (dict(N=0, x=None, w=None, hidden=None), OK), (dict(N=0, kind=2), OK),
])
def test_gated_validation(lib, kwargs, expect):
    assert gated(lib, **kwargs) == expect


def gated_backward(lib, dh=A, x=B, w=C_, saved=D, exps=None, off=E_, gx=F_, gw=G, hidden=H, N=40,
                   E=4, F=32, C=64, act=0, kind=1, ws=WS, wsb=1 << 20):
    return lib.latent_tail_expert_gated_backward(dh, x, w, saved, exps, off, gx, gw, hidden, N, E,
                                                 F, C, act, kind, ws, wsb, None)


@pytest.mark.parametrize("kwargs,expect", [
    (dict(N=-1), BAD), (dict(E=1025), BAD), (dict(C=60), ALIGN), (dict(F=32776), BAD),
    (dict(off=None), BAD), (dict(act=7), BAD), (dict(kind=0, saved=None), BAD),
    (dict(saved=None), BAD), (dict(kind=2), BAD), (dict(exps=I), BAD),
    (dict(gx=None, gw=None, hidden=None), BAD), (dict(dh=None), BAD), (dict(w=None), BAD),
    (dict(x=None), BAD), (dict(x=B + 2), ALIGN), (dict(gx=F_ + 4), ALIGN),
    (dict(ws=None), Status.WORKSPACE), (dict(wsb=40 * 128 - 1), Status.WORKSPACE),
    (dict(ws=WS + 4), ALIGN), (dict(gx=B), BAD), (dict(gw=C_ + 64), BAD), (dict(hidden=F_), BAD),
    (dict(ws=D + 128), BAD), (dict(hidden=A), BAD),
])
def test_gated_backward_validation(lib, kwargs, expect):
    assert gated_backward(lib, **kwargs) == expect


def test_gated_backward_workspace_size(lib):
    size = lib.latent_tail_expert_gated_backward_workspace_size
    assert size(40, 32) == 40 * 64 * 2
    assert size(1 << 24, 32768) == (1 << 24) * 65536 * 2
    assert size(0, 32) == size(-1, 32) == size(4, 36) == size(4, 32776) == size(4, 0) == 0


@pytest.mark.parametrize("kwargs,expect", SIZES + [
    (dict(M=4), BAD), (dict(M=65544), BAD), (dict(M=12), ALIGN), (dict(out=None), BAD),
    (dict(out=A + 16), BAD), (dict(out=D), BAD), (dict(N=0, x=None, w=None, out=None), OK),
])
def test_matmul_validation(lib, kwargs, expect):
    p = dict(x=A, w=B, off=D, out=C_, N=40, E=4, M=32, C=64)
    p.update(kwargs)
    args = [p[k] for k in ("x", "w", "off", "out", "N", "E", "M", "C")]
    assert lib.latent_tail_expert_matmul(*args, None) == expect
    assert lib.latent_tail_selftest_expert_matmul_timeout(*args, 0, 1000, None) == expect
    for copied, limit in ((-1, 1000), (0, 0), (0, 1000001)):
        assert lib.latent_tail_selftest_expert_matmul_timeout(*args, copied, limit, None) == BAD


@pytest.mark.parametrize("kwargs,expect", [
    (dict(N=-1), BAD), (dict(E=0), BAD), (dict(M=12), ALIGN), (dict(C=65544), BAD),
    (dict(off=None), BAD), (dict(dy=None), BAD), (dict(gx=None, gw=None), BAD),
    (dict(w=None), BAD), (dict(x=None), BAD), (dict(dy=A + 2), ALIGN), (dict(gw=F_ + 4), ALIGN),
    (dict(gx=A), BAD), (dict(gw=B), BAD), (dict(gw=E_ + 128), BAD), (dict(gx=D), BAD),
])
def test_matmul_backward_validation(lib, kwargs, expect):
    p = dict(dy=A, x=B, w=C_, off=D, gx=E_, gw=F_, N=40, E=4, M=32, C=64)
    p.update(kwargs)
    args = [p[k] for k in ("dy", "x", "w", "off", "gx", "gw", "N", "E", "M", "C")]
    assert lib.latent_tail_expert_matmul_backward(*args, None) == expect


@pytest.mark.parametrize("kwargs,expect", [
    (dict(T=-1), BAD), (dict(T=(1 << 24) + 1), BAD), (dict(C=0), BAD), (dict(C=65544), BAD),
    (dict(C=20), ALIGN), (dict(a=None), BAD), (dict(b=None), BAD), (dict(c=None), BAD),
    (dict(a=A + 8), ALIGN), (dict(b=B + 8), ALIGN), (dict(c=C_ + 1), ALIGN),
    (dict(T=0, a=None, b=None, c=None), OK),
])
def test_8_bit_validation(lib, kwargs, expect):
    p = dict(a=A, b=B, c=C_, T=10, C=72)
    p.update(kwargs)
    args = (p["a"], p["b"], p["c"], p["T"], p["C"], None)
    assert lib.latent_tail_quantize8(*args) == expect
    assert lib.latent_tail_dequantize8(*args) == expect


def test_8_bit_overlaps(lib):
    for q in ((A, A + 16, C_), (A, B, A + 32), (A, B, B + 16)):
        assert lib.latent_tail_quantize8(*q, 10, 72, None) == BAD
    for d in ((A, B, A + 16), (A, B, B)):
        assert lib.latent_tail_dequantize8(*d, 10, 72, None) == BAD


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda wide: lt.expert_gated(wide(8), meta(1, 16, 8)),
    lambda wide: lt.expert_matmul(wide(8), meta(1, 8, 8)),
    lambda wide: lt.expert_matmul_backward(wide(8), None, meta(1, 8, 8)),
    lambda wide: lt.expert_gated_backward(None, None, None, meta(2 ** 32 + 5, 2, 8)),
    lambda wide: lt.quantize8(wide(8)),
    lambda wide: lt.quantize8(meta(2 ** 17, 2 ** 15, 8)),
    lambda wide: lt.dequantize8(lt.Checkpoint8(wide(8), wide(1)))])
def test_sizes_that_a_c_int_does_not_hold_are_refused(call):
    with pytest.raises(ValueError, match="at most 2147483647"):
        call(lambda n: meta(2 ** 32 + 5, n))


def test_python_refusals():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        lt.expert_gated(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        lt.expert_matmul(x[0], w)
    with pytest.raises(TypeError):
        lt.expert_matmul(None, w)
    with pytest.raises(ValueError, match="both None"):
        _both_none()
    with pytest.raises(ValueError, match="activation"):
        lt.expert_gated_backward(x, x, w, meta(4, 2, 8), activation="relu")
    with pytest.raises(ValueError, match="save"):
        lta.expert_ffn(x, w, w, save="4bit")
    with pytest.raises(ValueError, match="dimensions"):
        lt.quantize8(torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        lt.expert_gated_backward(x, x, w, meta(4, 3, 8))


def _both_none():
    """The check stands before the one for the device of x and weights."""
    from unittest import mock

    from latent_moe_output_gb300 import experts

    with mock.patch.object(experts, "_index", return_value=0):
        return experts.expert_matmul_backward(torch.zeros(4, 8, dtype=torch.bfloat16), None, None)


# ------------------------------------------------------ the 8-bit reference itself
def test_8_bit_reference():
    """Half a unit, and a unit of at most 1/63.5 of the largest magnitude of the group."""
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(64, 40, generator=g) * torch.exp(6 * torch.randn(64, 1, generator=g))
         ).to(torch.bfloat16).double()
    x[0, :16] = 0
    x[1, 3], x[2, 20], x[3, 39] = float("inf"), float("nan"), float("-inf")
    x[4, :16] = 127.5 * 2.0 ** 5
    x[5, :16] = 127.0 * 2.0 ** 5
    q, e = er.quantize8(x)
    y = er.dequantize8(q, e)
    assert e[0, 0] == 0 and e[1, 0] == e[2, 1] == e[3, 2] == 255
    assert e[4, 0] == 127 + 6 and e[5, 0] == 127 + 5 and q[5, 0] == 127
    for a in range(0, 40, 16):
        part, back = x[:, a:a + 16], y[:, a:a + 16]
        ok = torch.isfinite(part).all(-1)
        top = part[ok].abs().amax(-1, keepdim=True)
        assert ((part[ok] - back[ok]).abs() <= top / 127).all()
        assert torch.isnan(back[~ok]).all()
    assert torch.equal(y[torch.isfinite(y).all(-1)],
                       y[torch.isfinite(y).all(-1)].to(torch.bfloat16).double())
