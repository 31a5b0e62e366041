"""Temperatures at the end of the range: refused where log2(e) / temperature is infinite in fp32,
which gave NaN for every row (no GPU needed: the calls below fail validation, or want a workspace)."""
import pytest

from lora_rank_adapter_gb300 import training
from tests.test_training_host import INVALID, L, logps, logps_bwd, policy, pref  # noqa: F401


@pytest.mark.parametrize("temperature", [3e-39, 4.2e-39])
def test_refused(L, temperature):  # noqa: F811
    for call in (logps, logps_bwd, pref, policy):
        assert call(L, temp=temperature, V=training.POLICY_HELD_BYTES // 2 + 1, ld=1 << 20) == INVALID, call.__name__


def test_the_smallest_that_is_taken(L):  # noqa: F811
    assert logps(L, T=0, temp=4.3e-39, x=None, lab=None, out=None) == 0
    assert logps(L, T=0, temp=3e38, x=None, lab=None, out=None) == 0
