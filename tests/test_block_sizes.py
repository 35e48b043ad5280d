"""Sizes of the operators around the tail that their C entry points cannot be given."""

import pytest
import torch

import latent_moe_output_gb300 as lt


@pytest.mark.parametrize("call", [
    lambda wide: lt.dispatch(None, wide(2, torch.int32), 8),
    lambda wide: lt.combine(wide(8), wide(2, torch.int32)),
    lambda wide: lt.combine_backward(wide(8), None, wide(2, torch.int32)),
    lambda wide: lt.expert_matvec4(wide(32), *(torch.empty(1, 8, n, device="meta")
                                               for n in (16, 1))),
    lambda wide: lt.residual_norm(wide(8), wide(8), None, None, 1e-6),
    lambda wide: lt.residual_norm_backward(wide(8), None, wide(8), wide(8), None, None, 1e-6),
    lambda wide: lt.dispatch(None, torch.empty(4, 2, dtype=torch.int32, device="meta"),
                             2 ** 32 + 8)])
def test_sizes_that_a_c_int_does_not_hold_are_refused(call):
    """2^32 + 5 tokens would arrive as 5."""
    def wide(n, dtype=torch.bfloat16):
        return torch.empty(2 ** 32 + 5, n, dtype=dtype, device="meta")

    with pytest.raises(ValueError, match="at most 2147483647"):
        call(wide)
