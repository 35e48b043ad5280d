"""Edges of the operators around the tail on the GPU: rows that no expert owns,
orders of summation, waits that expire."""

import pytest
import torch

import latent_moe_output_gb300 as lt
from latent_moe_output_gb300.binding import latent_tail_check

import block_reference as br
import gpu_helpers as gh
from test_gpu_block import gen, randn, weights4

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
