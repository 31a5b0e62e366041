"""What the optimizer takes over, by memory layout (on the CPU)."""
from types import SimpleNamespace

import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops, training

E4M3 = torch.float8_e4m3fn


def _optimizer(p, **k):
    return torch_ops.AdamW([p.requires_grad_()], **k)


def _filled(opt):
    g = torch.Generator().manual_seed(0)
    for values in opt._states().values():
        for t in values:
            t.copy_(torch.rand(t.shape, generator=g).to(t.dtype))
    return opt


def _same(a, b):
    return all(torch.equal(t.float(), u.float()) for k in a if k != "step" for t, u in zip(a[k], b[k]))


def test_8_bit_codes_of_another_layout_are_refused():
    """Codes copied element by element between layouts would meet the scales of other elements."""
    transposed = lambda: torch.zeros(24, 40).t()  # noqa: E731
    saved = _filled(_optimizer(transposed(), state_bits=8)).state_dict()
    assert saved["exp_avg"][0].stride() == (1, 40)
    target = _optimizer(torch.zeros(40, 24), state_bits=8)
    before = target.state_dict()
    with pytest.raises(ValueError, match="layout"):
        target.load_state_dict(saved)
    assert _same(target.state_dict(), before)
    same = _optimizer(transposed(), state_bits=8)
    same.load_state_dict(saved)
    assert _same(same.state_dict(), saved)
    # strides of axes of one element say nothing
    column = _filled(_optimizer(torch.zeros(1, 40).t(), state_bits=8)).state_dict()
    other = _optimizer(torch.zeros(40, 1), state_bits=8)
    other.load_state_dict(column)
    assert _same(other.state_dict(), column)


def test_32_bit_states_and_masters_are_taken_by_element():
    saved = _filled(_optimizer(torch.zeros(24, 40).t(), masters=True)).state_dict()
    target = _optimizer(torch.zeros(40, 24), masters=True)
    target.load_state_dict(saved)
    assert _same(target.state_dict(), saved)


def test_states_are_not_replaced_under_the_plan():
    """A plan holds addresses: a tensor put in a state's place would leave the step writing to the
    memory of the one that is gone."""
    opt = _optimizer(torch.zeros(4, 4), state_bits=8, masters=True)
    for name in ("params", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale", "masters"):
        with pytest.raises(TypeError):
            getattr(opt, name)[0] = torch.zeros(4, 4)


def test_tensors_without_elements_are_dense():
    for t in (torch.zeros(5, 0), torch.zeros(0, 5), torch.zeros(0, 5).t(), torch.zeros(0), torch.zeros(3, 0, 2),
              torch.zeros(4, 6)[:, :0], torch.zeros(4, 6)[::2, 3:3]):
        assert training._dense(t), (t.shape, t.stride())
    assert not training._dense(torch.zeros(4, 6)[:, :5]) and training._dense(torch.zeros(()))


@pytest.mark.gpu
def test_a_plan_skips_tensors_without_elements():
    dev = "cuda:0"
    torch.cuda.set_device(0)
    shapes = [(5, 0), (7, 3), (0, 4)]
    make = lambda: [torch.ones(s, device=dev) for s in shapes]  # noqa: E731
    s = SimpleNamespace(p=make(), g=make(), m=make(), v=make())
    plan = training.lora_adamw_plan(s.p, s.g, s.m, s.v)
    norm = torch.empty(2, device=dev)
    training.lora_grad_norm(plan, 1.0, norm)
    assert abs(float(norm[0]) - 21 ** 0.5) < 1e-5
    training.lora_adamw(plan, lr=0.1, step=1)
    assert bool((s.p[1] != 1).all())
