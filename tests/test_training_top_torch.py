"""top_logps and distill_loss in torch: fake implementations and second derivatives on the CPU, autograd
against plain torch in 64 bits, and both together as they are used, a teacher's record and a student's step.

Tolerances: logits of a spread of 2 over 203 columns, |ln p| below 20, so log-probabilities and
entropies are off by 4e-6 * 20 at most and gradients by 1e-4 of their largest element in fp32, with
a rounding of 2^-8 in bf16."""
import importlib.util
import math
import os

import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops, training
from tests._util import ROOT

DEV = "cuda:0"
TOL = {torch.float32: 1e-4, torch.bfloat16: 2.0 ** -8}


def test_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x, labels = torch.empty((10, 50), dtype=torch.bfloat16), torch.empty((10,), dtype=torch.int64)
        out = torch.ops.lora_gb300.top_logps(x, labels, 7, 1.0)
        assert [tuple(t.shape) for t in out] == [(10, 7), (10, 7), (10,), (10,), (10,), (10, 2)]
        assert out[0].dtype == torch.int64 and all(t.dtype == torch.float32 for t in out[1:])
        assert torch.ops.lora_gb300.top_logps(x, None, 7, 1.0)[4].shape == (0,)
        d = torch.ops.lora_gb300.top_logps_backward(x, None, out[0], out[5], out[2], None, out[2], out[1], 1.0)
        assert d.shape == x.shape and d.dtype == x.dtype
        top = x.new_empty((10, 7), dtype=torch.float32)
        for wanted, shape in ((True, (10, 50)), (False, (0, 0))):
            out = torch.ops.lora_gb300.distill_loss(x, out[0] if wanted else ids, top, None, None, "forward", 1.0, wanted)
            assert [tuple(t.shape) for t in out] == [(), (10,), shape]
            ids = labels[:, None].expand(10, 7)


def _inputs(dtype, T=14, V=203, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V, generator=g) * 2).to(dtype)
    labels = torch.randint(0, V, (T,), generator=g)
    labels[[0, 5]] = -100
    return x, labels


def _close(got, want, tol):
    assert float((got.double().cpu() - want).abs().max()) <= tol * float(want.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("use", ["logps", "entropy", "label_logps", "all", "none"])
def test_autograd_of_top_logps(dtype, use):
    x, labels = _inputs(dtype)
    T, K, temp = 14, 9, 0.9
    g = torch.Generator().manual_seed(1)
    a, b, c = torch.randn(T, K, generator=g), torch.randn(T, generator=g), torch.randn(T, generator=g)
    z = x.double().requires_grad_(True)
    lnp = torch.log_softmax(z / temp, 1)
    ok = labels >= 0
    order = torch.sort(x.double(), dim=1, descending=True, stable=True)[1][:, :K]
    parts = {"logps": (lnp.gather(1, order) * a)[ok].sum(), "entropy": (-(lnp.exp() * lnp).sum(1) * b)[ok].sum(),
             "label_logps": (lnp[torch.arange(T), labels.clamp(min=0)] * c)[ok].sum()}
    mine = x.to(DEV).requires_grad_(True)
    out = torch_ops.top_logps(mine, K, labels.to(DEV), temp)
    assert torch.equal(out.ids.cpu()[ok], order[ok]) and not out.ids.requires_grad and not out.rest.requires_grad
    rows = ok.to(DEV)
    got = {"logps": (out.logps * a.to(DEV))[rows].sum(), "entropy": (out.entropy * b.to(DEV)).sum(),
           "label_logps": (out.label_logps * c.to(DEV)).sum()}
    if use == "none":
        assert torch_ops.top_logps(mine, K).label_logps is None
        return
    chosen = list(parts) if use == "all" else [use]
    want, = torch.autograd.grad(sum(parts[k] for k in chosen), z)
    loss = sum(got[k] for k in chosen)
    assert abs(float(loss.detach()) - float(sum(parts[k] for k in chosen).detach())) <= 8e-5 * T * K
    loss.backward()
    _close(mine.grad, want, TOL[dtype])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["forward", "reverse"])
@pytest.mark.parametrize("with_rest", [True, False])
def test_autograd_of_distill_loss(dtype, kind, with_rest):
    """From a record that top_logps made of a teacher's logits; weights None are the mean."""
    x, _ = _inputs(dtype)
    teacher, _ = _inputs(dtype, seed=4)
    T, K, temp, factor = 14, 9, 0.9, -2.5
    record = torch_ops.top_logps(teacher.to(DEV), K, temperature=temp)
    q = torch.log_softmax(teacher.double() / temp, 1)
    ids = torch.sort(teacher.double(), dim=1, descending=True, stable=True)[1][:, :K]
    assert torch.equal(record.ids.cpu(), ids)
    z = x.double().requires_grad_(True)
    p = torch.log_softmax(z / temp, 1)
    listed = torch.zeros(T, 203, dtype=torch.bool).scatter_(1, ids, True)
    lnp, lnq = p.gather(1, ids), q.gather(1, ids)
    if with_rest:
        others = lambda v: v.masked_fill(listed, -math.inf).logsumexp(1, keepdim=True)  # noqa: E731
        lnp, lnq = torch.cat([lnp, others(p)], 1), torch.cat([lnq, others(q)], 1)
    rows = ((lnq.exp() * (lnq - lnp)) if kind == "forward" else (lnp.exp() * (lnp - lnq))).sum(1)
    want, = torch.autograd.grad(rows.mean() * factor, z)
    mine = x.to(DEV).requires_grad_(True)
    loss, row_loss = torch_ops.distill_loss(mine, record.ids, record.logps, record.rest if with_rest else None, kind=kind,
                                            temperature=temp)
    assert not row_loss.requires_grad and abs(float(loss.detach()) - float(rows.mean().detach())) <= 2e-4
    (loss * factor).backward(retain_graph=True)
    # a factor that is no power of two rounds the bf16 gradient once more
    _close(mine.grad, want, TOL[dtype] * (2 if dtype == torch.bfloat16 else 1))
    with pytest.raises(RuntimeError, match="once"):
        loss.backward()
    with torch.no_grad():
        quiet, _ = torch_ops.distill_loss(mine, record.ids, record.logps, kind=kind, temperature=temp)
    assert not quiet.requires_grad


@pytest.mark.gpu
def test_opcheck():
    x, labels = _inputs(torch.float32)
    x, labels = x.to(DEV), labels.to(DEV)
    check = lambda op, args: torch.library.opcheck(op, args, test_utils=("test_schema", "test_faketensor"))  # noqa: E731
    check(torch.ops.lora_gb300.top_logps, (x, labels, 5, 1.0))
    check(torch.ops.lora_gb300.top_logps, (x, None, 0, 0.7))
    ids, top, entropy, rest, logps, stats = torch.ops.lora_gb300.top_logps(x, labels, 5, 1.0)
    check(torch.ops.lora_gb300.top_logps_backward, (x, labels, ids, stats, entropy, logps, entropy, top.exp(), 1.0))
    check(torch.ops.lora_gb300.distill_loss, (x, ids, top, rest, None, "reverse", 1.0, True))


def _distill_formula(logits, ids, top, rest, weights, kind, temperature, wanted):
    with torch.no_grad():
        lnp = torch.log_softmax(logits, 1)
        d = torch.zeros_like(logits).scatter_(1, ids, -top.exp()) + lnp.exp() * top.exp().sum(1, keepdim=True)
        loss = -(top.exp() * lnp.gather(1, ids)).sum()
    return [loss, torch.zeros(len(ids)), d if wanted else logits.new_empty((0, 0))]


@pytest.mark.parametrize("gpu", [False, pytest.param(True, marks=pytest.mark.gpu)])
def test_second_derivatives_of_the_distillation_loss_raise(gpu, monkeypatch):
    """On the CPU with the kernels replaced by the formula."""
    device = DEV if gpu else "cpu"
    if not gpu:
        monkeypatch.setattr(torch_ops, "distill_loss_op", _distill_formula)
        monkeypatch.setattr(training, "lora_scale_gradient", lambda d, f: d.mul_(f))
    g = torch.Generator().manual_seed(0)
    x, W = torch.randn(6, 3, generator=g).to(device), torch.randn(3, 7, generator=g).to(device).requires_grad_()
    ids = torch.tensor([[1, 0], [4, 2], [2, 1], [0, 6], [5, 3], [3, 4]], device=device)
    top = torch.log(torch.full((6, 2), 0.4)).to(device)
    loss = lambda: torch_ops.distill_loss(torch.tanh(x @ W), ids, top)[0]  # noqa: E731
    (dW,) = torch.autograd.grad(loss(), W, create_graph=True)
    (first,) = torch.autograd.grad(loss(), W)
    assert torch.equal(dW.detach(), first) and not first.requires_grad
    with pytest.raises(RuntimeError, match="second derivatives|no autograd formula"):
        torch.autograd.grad(dW.square().sum(), W)


@pytest.mark.gpu
def test_second_derivatives_of_top_logps_raise():
    g = torch.Generator().manual_seed(0)
    x, W = torch.randn(6, 3, generator=g).to(DEV), torch.randn(3, 7, generator=g).to(DEV).requires_grad_()
    out = torch_ops.top_logps(torch.tanh(x @ W), 2)
    (dW,) = torch.autograd.grad(out.entropy.sum() + out.logps.sum(), W, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives|no autograd formula"):
        torch.autograd.grad(dW.square().sum(), W)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_record_and_steps_on_it(dtype):
    """Teacher's logits -> record -> student's loss and gradient through an adapter -> AdamW, and the same
    with the gradient of the formula in 64 bits: the adapters' gradients agree."""
    g = torch.Generator().manual_seed(3)
    T, wide, V, r, K = 40, 32, 304, 8, 16
    h, base = torch.randn(T, wide, generator=g).to(dtype), torch.randn(T, V, generator=g).to(dtype)
    A, B = (torch.randn(wide, r, generator=g) / 4).to(dtype), (torch.randn(r, V, generator=g) / 4).to(dtype)
    on = lambda t: t.to(DEV)  # noqa: E731
    record = torch_ops.top_logps(on(base), K)
    a, b = on(A).requires_grad_(True), on(B).requires_grad_(True)
    opt = torch_ops.AdamW([a, b], lr=1e-2)
    logits = torch_ops.lora_linear(on(h), a, b, on(base), 2.0)
    logits.retain_grad()
    loss, _ = torch_ops.distill_loss(logits, record.ids, record.logps, record.rest)
    loss.backward()
    z = logits.detach().double().cpu().requires_grad_(True)
    p = torch.log_softmax(z, 1)
    ids, lnq = record.ids.cpu(), record.logps.double().cpu()
    listed = torch.zeros(T, V, dtype=torch.bool).scatter_(1, ids, True)
    lnp = torch.cat([p.gather(1, ids), p.masked_fill(listed, -math.inf).logsumexp(1, keepdim=True)], 1)
    lnq = torch.cat([lnq, record.rest.double().cpu()[:, None]], 1)
    (lnq.exp() * (lnq - lnp)).sum(1).mean().backward()
    _close(logits.grad, z.grad, TOL[dtype])
    d = logits.grad.double().cpu()
    # fp32: sums of 40 and 304 products; bf16: the result's rounding
    _close(a.grad, 2 * h.double().t() @ (d @ B.double().t()), 2e-5 if dtype == torch.float32 else 2.0 ** -7)
    _close(b.grad, 2 * (h.double() @ A.double()).t() @ d, 2e-5 if dtype == torch.float32 else 2.0 ** -7)
    before = a.detach().clone()
    opt.step()
    assert bool((a.detach() != before).any()) and bool(a.isfinite().all()) and bool(b.isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("args", [["--loss", "distill"], ["--loss", "policy", "--entropy-bonus", "0.01"]])
def test_example_runs(args):
    spec = importlib.util.spec_from_file_location("preference_finetune",
                                                  os.path.join(ROOT, "examples", "preference_finetune.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.main(args + ["--steps", "4"])
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
