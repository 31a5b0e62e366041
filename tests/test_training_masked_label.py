"""The policy loss on the policy itself (no old_logps: r = 1) where a label is masked out by minus
infinity: the row counts like any other, and its gradient is that of its log-probability,
-A w (onehot - p) with a probability of 0 at the label."""
import math

import pytest
import torch

from tests.test_training_loss import BF16, DEV, F32, check_dlogits, make, oracle_dlogits, oracle_logps, run_policy


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(9, 40), (9, 2500), (9, 40001), (2, 400000)])
def test_a_masked_label_on_the_policy_itself(T, V, dtype):
    torch.cuda.set_device(0)
    _, x, labels = make(T, V, dtype, seed=1, ignored=0.0)
    x[1, int(labels[1])] = -math.inf
    x[T - 1, V // 2:] = math.nan                # NaN stays NaN
    g = torch.Generator().manual_seed(2)
    adv, w = torch.randn(T, generator=g), torch.rand(T, generator=g)
    got = run_policy(x, labels, None, adv, w)
    _, p, ok = oracle_logps(x, labels)
    if T > 2:
        assert float(got["tok"][1]) == -math.inf
        coef = -(adv * w).double()
        rows = torch.arange(T - 1)
        check_dlogits(got["d"][rows.to(DEV)], oracle_dlogits(p, labels, ok, coef)[rows], coef[rows],
                      2e-6 * coef[rows].abs())
    assert bool(got["d"][T - 1].isnan().any()) and bool(got["metrics"][0].isnan())
    # without the NaN row the loss is the sum of -A w
    fine = run_policy(x[:T - 1], labels[:T - 1], None, adv[:T - 1], w[:T - 1])
    want = -float((adv.double() * w.double())[:T - 1].sum())
    assert abs(float(fine["metrics"][0]) - want) <= 1e-6 * float((adv.abs() * w).sum())
    assert float(fine["metrics"][1]) == 0.0 and float(fine["metrics"][2]) == 0.0
