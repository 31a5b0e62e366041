"""Workspaces that a caller passes in: one that the kernels could not write whole is refused
before the call (the library replaced, no GPU needed)."""
import pytest
import torch

from lora_rank_adapter_gb300 import training
from tests.test_other_gpu_host import I32, I64, Far, gpus  # noqa: F401


def _preference(ws):
    T, V = 6, 40
    return training.lora_preference_loss(Far(T, V), Far(T, dtype=I64), Far(3, dtype=I32), None, 0.1, Far(T), Far(2), Far(1),
                                         Far(1), ws=ws)


def _policy(ws):
    T, V = 2, 200000      # 800 KB a row: past what is held on chip
    return training.lora_policy_loss(Far(T, V), Far(T, dtype=I64), None, Far(T), None, Far(T), Far(3), dlogits=Far(T, V), ws=ws)


@pytest.mark.parametrize("call", [_preference, _policy])
def test_a_workspace_off_the_gpu_or_with_gaps_is_refused(gpus, call):  # noqa: F811
    _, calls = gpus
    gaps = Far(8192, dtype=torch.uint8)
    gaps.is_contiguous = lambda: False
    here = Far(8192, dtype=torch.uint8)
    here.get_device = lambda: 0
    for ws in (torch.empty(8192, dtype=torch.uint8), gaps, here):
        with pytest.raises(ValueError, match="ws"):
            call(ws)
    assert not calls
    call(Far(8192, dtype=torch.uint8))
    assert len(calls) == 1


def test_a_workspace_counts_in_bytes(gpus, monkeypatch):  # noqa: F811
    sizes = []

    class Library:
        def lora_preference_loss(self, *args):
            sizes.append(args[-2])
            return 0

    monkeypatch.setattr(training, "lib", lambda: Library())
    _preference(Far(1000))
    assert sizes == [4000]
