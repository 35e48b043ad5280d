"""The workloads of perf/operators.py: their plain torch forms and the package's operators
against their 64-bit definitions, on the listed cases of up to about 1000 tokens.

Bound, for the norm of a tensor's error against the norm of its exact value: a bf16 value
is off by at most 2^-8 of itself, and FP32 sums of up to 1024 random terms by
(256 + 1024) * 2^-24 of the terms' magnitudes, about 32 times the sum: 2.5e-3 < 2^-8."""

import importlib.util
from pathlib import Path

import pytest
import torch

import gpu_helpers as gh

pytestmark = pytest.mark.gpu

_spec = importlib.util.spec_from_file_location(
    "operator_workloads", Path(__file__).resolve().parents[1] / "perf" / "operators.py")
workloads = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(workloads)
CASES = [c for c in workloads.listed() if c["T"] <= 1024]


@pytest.fixture(scope="module", autouse=True)
def lib():
    return gh.library()


def parts(v):
    return list(v) if isinstance(v, (tuple, list)) else [v]


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c["name"] for c in CASES])
def test_workload_against_its_definition(case, own, monkeypatch):
    monkeypatch.setattr(workloads, "own", own)
    got = parts(workloads.run(workloads.prepare(case, 11)))
    want = parts(workloads.exact(case, 11))
    assert len(got) == len(want)
    for i, (a, b) in enumerate(zip(got, want)):
        if b is None:
            assert a is None, i
        elif not b.is_floating_point():
            assert torch.equal(a, b), i
        else:
            assert a.shape == b.shape
            assert (a.double() - b).norm() <= 2.0 ** -8 * b.norm(), i
