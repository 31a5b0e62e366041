"""The optimizer's count of steps of each parameter: gradients that come late or now and then,
beside torch.optim.AdamW, which counts for each parameter too.  On the CPU with the library's
calls replaced by their formulas, on the GPU with the kernels."""
import math
from types import SimpleNamespace

import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops, training

DEV = "cuda:0"
SHAPES = [(33, 70), (513,), (4, 4), (300,)]


def has_gradient(i, step):
    """Parameter 0 at every step, 1 from step 30 on, 2 at two steps of three, 3 at every fifth."""
    return (True, step >= 30, step % 3 != 1, step % 5 == 4)[i]


def gradient(i, step):
    g = torch.Generator().manual_seed(100 * step + i)
    return torch.randn(SHAPES[i], generator=g) + 0.5


def run(opt, params, steps, device, clip=None):
    for step in steps:
        for i, p in enumerate(params):
            p.grad = gradient(i, step).to(device) if has_gradient(i, step) else None
        if clip is not None:
            torch.nn.utils.clip_grad_norm_(params, clip)
        opt.step()


def start(device):
    g = torch.Generator().manual_seed(7)
    return [torch.randn(s, generator=g).to(device).requires_grad_() for s in SHAPES]


def close(mine, ref, begin):
    """32-bit states: some roundings of 2^-24 a step of values and updates, 60 steps."""
    for i, (p, q, s) in enumerate(zip(mine, ref, begin)):
        off, way = (p - q).detach().norm(), (q - s).detach().norm()
        assert float(off) <= 2e-5 * float(way), i


def check(device, clip=None):
    begin, mine, ref = start(device), start(device), start(device)
    a = torch_ops.AdamW(mine, lr=1e-2, weight_decay=0.05, max_norm=clip)
    b = torch.optim.AdamW(ref, lr=1e-2, weight_decay=0.05)
    run(a, mine, range(31), device)
    run(b, ref, range(31), device, clip)
    # the first step of a parameter is one of lr along each sign, whenever it comes
    moved = (mine[1] - begin[1] * (1 - 1e-2 * 0.05)).detach()
    assert float((moved.abs() - 1e-2).abs().max()) < 1e-5
    # resumed on the way, with the counts of each parameter
    state = a.state_dict()
    assert state["step"] == [31, 1, 21, 6]
    c = torch_ops.AdamW(mine, lr=1e-2, weight_decay=0.05, max_norm=clip)
    c.load_state_dict(state)
    run(c, mine, range(31, 60), device)
    run(b, ref, range(31, 60), device, clip)
    close(mine, ref, begin)
    with pytest.raises(ValueError):
        c.load_state_dict({**state, "step": [1, 2]})


@pytest.fixture
def formulas(monkeypatch):
    def plan(params, grads, m, v, masters=None, exp_avg_scales=None, exp_avg_sq_scales=None, stream=None,
             stochastic=False):
        assert masters is None and exp_avg_scales is None
        return SimpleNamespace(p=params, g=grads, m=m, v=v, tensors=None)

    def norm(plan, max_norm, out, stream=None):
        out[0] = math.sqrt(sum(float(g.double().square().sum()) for g in plan.g))
        out[1] = min(1.0, max_norm / (float(out[0]) + 1e-6))

    def step(plan, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_factor=None, stream=None):
        f = 1.0 if grad_factor is None else grad_factor[0]
        for p, g, m, v in zip(plan.p, plan.g, plan.m, plan.v):
            g = g * f
            m.copy_(beta1 * m + (1 - beta1) * g)
            v.copy_(beta2 * v + (1 - beta2) * g * g)
            p.copy_(p * (1 - lr * weight_decay) - lr / (1 - beta1 ** step) * m /
                    (v.sqrt() / math.sqrt(1 - beta2 ** step) + eps))

    monkeypatch.setattr(training, "lora_adamw_plan", plan)
    monkeypatch.setattr(training, "lora_grad_norm", norm)
    monkeypatch.setattr(training, "lora_adamw", step)


@pytest.mark.parametrize("clip", [None, 3.0])
def test_late_and_missing_gradients(formulas, clip):
    check("cpu", clip)


def test_one_count_where_all_step_together(formulas):
    params = start("cpu")
    opt = torch_ops.AdamW(params, lr=1e-2)
    for step in range(3):
        for i, p in enumerate(params):
            p.grad = gradient(i, step)
        opt.step()
        assert len(opt._groups) == 1
    assert opt.state_dict()["step"] == 3 and opt.step_count == 3
    again = torch_ops.AdamW(params, lr=1e-2)
    again.load_state_dict(opt.state_dict())
    assert again.step_count == 3 and again.state_dict()["step"] == 3


@pytest.mark.gpu
@pytest.mark.parametrize("clip", [None, 3.0])
def test_late_and_missing_gradients_on_the_gpu(clip):
    torch.cuda.set_device(0)
    check(DEV, clip)


@pytest.mark.gpu
@pytest.mark.parametrize("bits,masters", [(8, False), (8, True), (32, True)])
def test_resumed_with_counts_of_each_parameter(bits, masters):
    """The same codes and parameters, whether resumed or not."""
    torch.cuda.set_device(0)
    options = dict(lr=1e-2, state_bits=bits, masters=masters, max_norm=1.0)
    a, b = start(DEV), start(DEV)
    opt_a = torch_ops.AdamW(a, **options)
    run(opt_a, a, range(40), DEV)
    opt_b = torch_ops.AdamW(b, **options)
    run(opt_b, b, range(33), DEV)
    opt_c = torch_ops.AdamW(b, **options)
    opt_c.load_state_dict(opt_b.state_dict())
    run(opt_c, b, range(33, 40), DEV)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    counts = [sum(has_gradient(i, step) for step in range(40)) for i in range(4)]
    assert opt_c.state_dict()["step"] == opt_a.state_dict()["step"] == counts
