"""Host-side checks of the operators around the tail: bad arguments are refused
before any CUDA call, on a machine without a GPU too."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300 import binding
from latent_moe_output_gb300.binding import Status

import block_reference as br

# Fake, never-dereferenced addresses, 64 MiB apart.
A, B, C, D, E_, F, G_, H_, I, J, K_, L_, WS = (0x10000000 + 0x4000000 * i for i in range(13))


@pytest.fixture(scope="module")
def lib():
    from latent_moe_output_gb300 import build

    build.build()
    return binding.load_library()


def dispatch(lib, x=A, ids=B, rows=C, offsets=D, order=E_, position=F, T=1000, K=4, E=16, L=64,
             ws=WS, wsb=1 << 20):
    return lib.latent_tail_dispatch(x, ids, rows, offsets, order, position, T, K, E, L, ws, wsb,
                                    None)


@pytest.mark.parametrize("kwargs,expect", [
    (dict(T=-1), Status.INVALID_ARG),
    (dict(K=0), Status.INVALID_ARG),
    (dict(K=65), Status.INVALID_ARG),
    (dict(T=1 << 22, K=8), Status.INVALID_ARG),      # more than 2^24 choices
    (dict(E=0), Status.INVALID_ARG),
    (dict(E=1025), Status.INVALID_ARG),
    (dict(L=4), Status.INVALID_ARG),
    (dict(L=16392), Status.INVALID_ARG),
    (dict(L=60), Status.ALIGNMENT),
    (dict(x=None), Status.INVALID_ARG),              # rows without x
    (dict(rows=None), Status.INVALID_ARG),
    (dict(ids=None), Status.INVALID_ARG),
    (dict(offsets=None), Status.INVALID_ARG),
    (dict(order=E_ + 4), Status.ALIGNMENT),
    (dict(x=A + 2), Status.ALIGNMENT),
    (dict(ws=None), Status.WORKSPACE),
    (dict(wsb=64), Status.WORKSPACE),
    (dict(ws=WS + 8), Status.ALIGNMENT),
    (dict(rows=A + 64), Status.INVALID_ARG),         # overlaps x
    (dict(order=D + 16), Status.INVALID_ARG),        # two outputs overlap
    (dict(position=B), Status.INVALID_ARG),          # overlaps the ids
    (dict(ws=C + 256), Status.INVALID_ARG),
])
def test_dispatch_validation(lib, kwargs, expect):
    assert dispatch(lib, **kwargs) == expect


def test_dispatch_workspace_size(lib):
    size = lib.latent_tail_dispatch_workspace_size
    assert size(256, 8, 256) == 0            # one kernel, no workspace
    assert size(257, 8, 256) > 0
    assert size(1 << 22, 4, 1024) > 0
    assert size(0, 8, 256) == size(-1, 8, 256) == size(300, 65, 256) == size(300, 8, 1025) == 0


def test_combine_validation(lib):
    def call(rows=A, pos=B, w=C, out=D, T=10, K=4, L=64):
        return lib.latent_tail_combine(rows, pos, w, out, T, K, L, None)

    assert call(K=0) == Status.INVALID_ARG
    assert call(L=12) == Status.ALIGNMENT
    assert call(rows=None) == Status.INVALID_ARG
    assert call(w=C + 4) == Status.ALIGNMENT
    assert call(out=A + 128) == Status.INVALID_ARG
    assert call(T=0, rows=None, pos=None, out=None) == Status.OK

    def back(go=A, rows=B, pos=C, w=D, gr=E_, gw=F, T=10, K=4, L=64):
        return lib.latent_tail_combine_backward(go, rows, pos, w, gr, gw, T, K, L, None)

    assert back(rows=None) == Status.INVALID_ARG     # grad_weights needs the rows
    assert back(go=None) == Status.INVALID_ARG
    assert back(gr=B + 64) == Status.INVALID_ARG
    assert back(gw=F + 8) == Status.ALIGNMENT
    assert back(L=8 * 2049) == Status.INVALID_ARG
    assert back(T=0) == Status.OK


def test_matvec4_validation(lib):
    def call(x=A, q=B, s=C, off=D, out=E_, N=4, E=4, M=16, C_=64, G=32):
        return lib.latent_tail_expert_matvec4(x, q, s, off, out, N, E, M, C_, G, None)

    for kwargs, expect in [
        (dict(N=-1), Status.INVALID_ARG), (dict(E=0), Status.INVALID_ARG),
        (dict(E=1025), Status.INVALID_ARG), (dict(M=4), Status.INVALID_ARG),
        (dict(M=20), Status.ALIGNMENT), (dict(G=16), Status.INVALID_ARG),
        (dict(G=128), Status.INVALID_ARG),           # wider than C
        (dict(C_=96, G=64), Status.ALIGNMENT), (dict(C_=16416, G=32), Status.INVALID_ARG),
        (dict(off=None), Status.INVALID_ARG),        # several experts without offsets
        (dict(q=None), Status.INVALID_ARG), (dict(x=A + 8), Status.ALIGNMENT),
        (dict(off=D + 4), Status.ALIGNMENT), (dict(out=A + 16), Status.INVALID_ARG),
        (dict(N=0, x=None, out=None), Status.OK),
    ]:
        assert call(**kwargs) == expect, kwargs


def norm(lib, block=A, res=B, post=C, gate=D, nxt=E_, out=F, z=G_, T=4, H=64, kind=2, rt=0,
         scale=1.0, eps=1e-6):
    return lib.latent_tail_residual_norm(block, res, post, gate, nxt, out, z, T, H, kind, rt, scale,
                                         eps, None)


@pytest.mark.parametrize("kwargs,expect", [
    (dict(T=-1), Status.INVALID_ARG), (dict(H=4), Status.INVALID_ARG),
    (dict(H=16392), Status.INVALID_ARG), (dict(H=60), Status.ALIGNMENT),
    (dict(kind=4), Status.INVALID_ARG), (dict(kind=0), Status.INVALID_ARG),  # gate without a kind
    (dict(gate=None), Status.INVALID_ARG), (dict(rt=2), Status.INVALID_ARG),
    (dict(eps=0.0), Status.INVALID_ARG), (dict(eps=float("inf")), Status.INVALID_ARG),
    (dict(scale=float("inf")), Status.INVALID_ARG), (dict(block=None), Status.INVALID_ARG),
    (dict(z=None), Status.INVALID_ARG), (dict(nxt=None), Status.INVALID_ARG),
    (dict(post=C + 4), Status.ALIGNMENT), (dict(out=B + 16), Status.INVALID_ARG),
    (dict(z=B), Status.INVALID_ARG), (dict(out=A), Status.INVALID_ARG),
    (dict(z=F), Status.INVALID_ARG), (dict(T=0, block=None), Status.OK),
])
def test_residual_norm_validation(lib, kwargs, expect):
    assert norm(lib, **kwargs) == expect


@pytest.mark.parametrize("kwargs,expect", [
    (dict(gpost=None), Status.INVALID_ARG), (dict(gnext=None), Status.INVALID_ARG),
    (dict(dz=None), Status.INVALID_ARG), (dict(ggate=None), Status.INVALID_ARG),
    (dict(dv=None, dz=None, nxt=None, gnext=None), Status.INVALID_ARG),
    (dict(ws=None), Status.WORKSPACE), (dict(wsb=100), Status.WORKSPACE),
    (dict(ws=WS + 8), Status.ALIGNMENT), (dict(gblock=C), Status.INVALID_ARG),
    (dict(ws=I), Status.INVALID_ARG), (dict(gres=A), Status.INVALID_ARG),
    (dict(ggate=K_ + 4), Status.ALIGNMENT), (dict(H=12), Status.ALIGNMENT),
])
def test_residual_norm_backward_validation(lib, kwargs, expect):
    p = dict(dv=A, dz=B, block=C, out=D, post=E_, gate=F, nxt=G_, gblock=H_, gres=I, gpost=J,
             ggate=K_, gnext=L_, T=4, H=64, kind=2, rt=0, ws=WS, wsb=1 << 20)
    p.update(kwargs)
    st = lib.latent_tail_residual_norm_backward(
        p["dv"], p["dz"], p["block"], p["out"], p["post"], p["gate"], p["nxt"], p["gblock"],
        p["gres"], p["gpost"], p["ggate"], p["gnext"], p["T"], p["H"], p["kind"], p["rt"], 1.0,
        1e-6, p["ws"], p["wsb"], None)
    assert st == expect


def test_residual_norm_backward_workspace_size(lib):
    size = lib.latent_tail_residual_norm_backward_workspace_size
    assert size(1, 64) >= 2 * 64 * 4
    assert size(8192, 7168) >= 2 * 152 * 7168 * 4
    assert size(0, 64) == size(4, 60) == size(4, 16392) == 0


def test_tensors_in_host_memory_are_refused():
    x, ids = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        lt.dispatch(x, ids, 8)
    with pytest.raises(ValueError):
        lt.residual_norm(x, x, None, None, 1e-6)
    with pytest.raises(TypeError):
        lt.dispatch(x, ids.tolist(), 8)


def test_quantize4_packs_even_columns_low():
    w = torch.zeros(2, 32)
    w[0, 0], w[0, 1], w[1, 2] = 7.0, -7.0, 3.5
    packed, scales = lt.quantize4(w, 32)
    assert packed.shape == (1, 2, 16) and scales.shape == (1, 2, 1)
    assert packed[0, 0, 0].item() == 15 | (1 << 4) and packed[0, 0, 1].item() == 8 | (8 << 4)
    assert torch.equal(br.unpack4(packed, scales)[0], w.double())


def test_reference_forms_agree_with_torch_autograd():
    """The 64-bit combine gradient that the GPU tests compare with, against autograd."""
    g = torch.Generator().manual_seed(3)
    T, K, L = 5, 3, 16
    ids = torch.randint(-1, 4, (T, K), generator=g, dtype=torch.int32)
    order, position, offsets = br.dispatch(ids, 4)
    assert sorted(order.tolist()) == list(range(T * K)) and offsets[-1] == (ids >= 0).sum()
    rows = torch.randn(T * K, L, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(T, K, generator=g, dtype=torch.float64, requires_grad=True)
    go = torch.randn(T, L, generator=g, dtype=torch.float64)
    here = (position >= 0)
    out = (rows[position.clamp(min=0).long()] * (w * here)[..., None]).sum(1)
    ref, _ = br.combine(rows.detach(), position, w.detach())
    torch.testing.assert_close(out.detach(), ref, atol=1e-14, rtol=1e-14)
    (out * go).sum().backward()
    gr, gw, _ = br.combine_backward(go, rows.detach(), position, w.detach())
    torch.testing.assert_close(rows.grad, gr, atol=1e-14, rtol=1e-14)
    torch.testing.assert_close(w.grad, gw, atol=1e-13, rtol=1e-13)
