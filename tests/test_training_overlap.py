"""Outputs that are inputs, and tensors given twice."""
import ctypes

import pytest
import torch

from lora_rank_adapter_gb300 import _build, torch_ops, training

INVALID, WORKSPACE = 1, 4
A, B, C = (ctypes.c_void_p(v) for v in (0x10000, 0x20000, 0x30000))


@pytest.mark.parametrize("which", ["old", "ref", "advantages", "weights"])
def test_token_logps_over_an_input_are_refused(which):
    """On a row that would be a launch, were it not refused; the same call with an output of its own
    gets as far as the workspace."""
    _build.build()
    V = training.POLICY_HELD_BYTES // 2 + 1
    inputs = {"old": C, "ref": C, "advantages": C, "weights": C}

    def call(token_logps, **k):
        k = {**inputs, **k}
        return training.lib().lora_policy_loss(1, 2, V, A, V, A, k["old"], k["ref"], k["advantages"], k["weights"], 0.2,
                                               0.2, 0.1, 1.0, token_logps, A, A, V, 1.0, None, 0, None)

    assert call(B) == WORKSPACE
    assert call(B, **{which: B}) == INVALID


def test_a_parameter_given_twice_is_refused():
    a, b = torch.zeros(4, requires_grad=True), torch.zeros(4, requires_grad=True)
    with pytest.raises(ValueError, match="twice"):
        torch_ops.AdamW([a, b, a])
    assert len(torch_ops.AdamW(p for p in (a, b)).params) == 2
