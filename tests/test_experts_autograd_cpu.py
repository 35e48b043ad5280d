"""What the autograd form of the gated block keeps, with the operators' calls replaced by
plain ones that write down what they are given (no GPU)."""

import contextlib
import types

import pytest
import torch

from latent_moe_output_gb300 import autograd as lta
from latent_moe_output_gb300 import experts


@pytest.fixture
def calls(monkeypatch):
    seen = types.SimpleNamespace(saved=[], quantized=0)

    def gated(x, up, offsets=None, activation="silu", saved=None):
        seen.saved.append(saved)
        gate, u = (x.float() @ up[0].float().t()).chunk(2, dim=1)
        return (torch.nn.functional.silu(gate) * u).to(x.dtype)

    def matmul(x, weights, offsets=None):
        return (x.float() @ weights[0].float().t()).to(x.dtype)

    def quantize8(x):
        seen.quantized += 1
        return experts.Checkpoint8.empty(*x.shape, device=x.device)

    for name, fn in (("expert_gated", gated), ("expert_matmul", matmul),
                     ("quantize8", quantize8)):
        monkeypatch.setattr(experts, name, fn)
    return seen


def tensors(*requires_grad):
    shapes = ((4, 16), (1, 32, 16), (1, 24, 16))
    return [torch.ones(*s, dtype=torch.bfloat16, requires_grad=r)
            for s, r in zip(shapes, requires_grad)]


@pytest.mark.parametrize("save", ["bf16", "8bit", "all8bit"])
@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_where_no_gradient_can_be_asked_for(calls, mode, save):
    """An evaluation pass of a block that is being trained."""
    args = tensors(True, True, True)
    with mode():
        out = lta.expert_ffn(*args, save=save)
    assert not out.requires_grad
    assert calls.saved == [None] and calls.quantized == 0


@pytest.mark.parametrize("save", ["bf16", "8bit", "all8bit"])
def test_nothing_is_kept_of_tensors_without_gradients(calls, save):
    lta.expert_ffn(*tensors(False, False, False), save=save)
    assert calls.saved == [None] and calls.quantized == 0


@pytest.mark.parametrize("save,kind,quantized", [("bf16", torch.Tensor, 0), ("8bit", tuple, 0),
                                                 ("all8bit", tuple, 1)])
@pytest.mark.parametrize("mode", [contextlib.nullcontext, torch.enable_grad])
def test_what_is_kept_for_a_backward_pass(calls, mode, save, kind, quantized):
    with torch.no_grad() if mode is torch.enable_grad else contextlib.nullcontext(), mode():
        out = lta.expert_ffn(*tensors(True, True, True), save=save)
    assert out.requires_grad
    assert isinstance(calls.saved[0], kind) and calls.quantized == quantized


def test_bits_are_given_up_only_where_the_caller_says_so(calls):
    lta.expert_ffn(*tensors(True, True, True))
    assert calls.saved[0].dtype == torch.bfloat16 and calls.quantized == 0


def test_the_training_example_keeps_bf16_unless_told_otherwise(calls, monkeypatch):
    """(its other operators replaced by ones that pass their input on)"""
    import importlib.util
    from pathlib import Path

    spec = importlib.util.spec_from_file_location(
        "latent_moe_block_cpu",
        Path(__file__).resolve().parents[1] / "examples" / "latent_moe_block.py")
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    monkeypatch.setattr(lta, "dispatch_rows",
                        lambda x, ids, E: types.SimpleNamespace(rows=x, offsets=None, position=ids))
    monkeypatch.setattr(lta, "combine_rows", lambda rows, position, weights: rows)
    monkeypatch.setattr(lta, "residual_norm",
                        lambda out, residual, post, nxt, eps, gate, residual_scale: (out, out))
    x, up, down = tensors(True, True, True)
    w = dict(up=up, down=down, latent_norm=torch.ones(24), post=None, next=None, gate=None,
             W=torch.ones(40, 24, dtype=torch.bfloat16))
    args = (w, x, None, None, torch.zeros(4, 40, dtype=torch.bfloat16), None)
    example.train_step(*args)
    example.train_step(*args, save="8bit")
    assert isinstance(calls.saved[0], torch.Tensor) and calls.saved[0].dtype == torch.bfloat16
    assert isinstance(calls.saved[1], tuple)
