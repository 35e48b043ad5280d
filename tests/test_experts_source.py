"""What the sources of the experts' kernels must not hold (no GPU, no build)."""

import re
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "latent_moe_output_gb300" / "csrc"


def code(name):
    """A source file without its comments."""
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


@pytest.mark.parametrize("name", ["experts.cu", "experts.cuh", "experts_few.cu", "quant8.cu"])
def test_no_load_may_move_above_the_wait_for_the_kernel_before(name):
    """These kernels start while the one before may still be writing their inputs. __ldg says
    that nothing does, so a compiler may issue it before the wait."""
    assert "__ldg" not in code(name)


def test_load_helpers_are_volatile():
    """... and the helpers that the kernels load with keep their place behind the wait."""
    text = code("ptx.cuh")
    found = 0
    for asm in re.findall(r"asm(?: volatile)?\s*\(\s*\"ld\.global[^;]*;", text):
        assert asm.startswith("asm volatile"), asm
        found += 1
    assert found >= 3
    assert re.search(r"pdl_wait\(\) \{ asm volatile\(\"griddepcontrol\.wait;\" ::: \"memory\"\)",
                     text)
