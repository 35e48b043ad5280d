"""Host-side edges of the operators around the tail, on a machine without a GPU too."""

import pytest

from latent_moe_output_gb300 import binding
from latent_moe_output_gb300.binding import Status

# Fake, never-dereferenced addresses, 64 MiB apart.
BLOCK, RES, POST, GATE, NEXT, OUT, Z = (0x10000000 + 0x4000000 * i for i in range(7))


@pytest.fixture(scope="module")
def lib():
    from latent_moe_output_gb300 import build

    build.build()
    return binding.load_library()


# ------------------------------------------ in place: the residual alone
@pytest.mark.parametrize("T,H,rt", [(1, 64, 1), (2, 64, 0)])  # residual of a vector's bytes
@pytest.mark.parametrize("name", ["post", "gate", "next"])
def test_residual_out_on_a_vector_that_is_the_residual_too_is_refused(lib, T, H, rt, name):
    """residual_out may be exactly residual. Where a weight or a channel gate is that same
    array too, it would be read after it was written."""
    p = dict(post=POST, gate=GATE, next=NEXT)
    p[name] = RES
    st = lib.latent_tail_residual_norm(BLOCK, RES, p["post"], p["gate"], p["next"], RES, Z, T, H,
                                       2, rt, 1.0, 1e-6, None)
    assert st == Status.INVALID_ARG
