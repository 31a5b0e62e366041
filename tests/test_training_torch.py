"""The training operators in torch: fake implementations on the CPU, autograd against plain
torch in 64 bits, the optimizer class, and the example that runs them together."""
import importlib.util
import math
import os

import pytest
import torch

from lora_rank_adapter_gb300 import torch_ops
from tests._util import ROOT

DEV = "cuda:0"


def test_fake_shapes():
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        x = torch.empty((10, 50), dtype=torch.bfloat16)
        labels = torch.empty((10,), dtype=torch.int64)
        logps, stats = torch.ops.lora_gb300.token_logps(x, labels, 1.0)
        assert logps.shape == (10,) and stats.shape == (10, 2) and logps.dtype == torch.float32
        d = torch.ops.lora_gb300.token_logps_backward(x, labels, stats, logps, 1.0)
        assert d.shape == x.shape and d.dtype == x.dtype
        cu = torch.empty((5,), dtype=torch.int32)
        out = torch.ops.lora_gb300.preference_loss(x, labels, cu, None, 0.1, "sigmoid", 0.0, False, 1.0, True)
        assert [tuple(t.shape) for t in out] == [(), (2,), (4,), (10,), (10, 50)]
        out = torch.ops.lora_gb300.preference_loss(x, labels, cu, None, 0.1, "sigmoid", 0.0, False, 1.0, False)
        assert tuple(out[4].shape) == (0, 0)
        out = torch.ops.lora_gb300.policy_loss(x, labels, None, logps, None, None, 0.2, 0.2, 0.0, 1.0, True)
        assert [tuple(t.shape) for t in out] == [(3,), (10,), (10, 50)]


def _inputs(dtype, T=14, V=203, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V, generator=g) * 2).to(dtype)
    labels = torch.randint(0, V, (T,), generator=g)
    labels[[0, 5]] = -100
    return x, labels


def _plain_logps(x, labels, temperature=1.0):
    p = torch.log_softmax(x.double() / temperature, 1)
    ok = labels >= 0
    return torch.where(ok, p[torch.arange(len(labels)), labels.clamp(min=0)], 0.0)


# fp32: some roundings of 2^-24 of sums of 14 tokens; bf16: the gradient's own rounding, 2^-9
TOL = {torch.float32: 2e-5, torch.bfloat16: 2.0 ** -8}


def _close(got, want, tol):
    assert float((got.double().cpu() - want).abs().max()) <= tol * float(want.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("factor", [1.0, -2.5])
def test_autograd(dtype, factor):
    x, labels = _inputs(dtype)
    cu = [0, 4, 7, 11, 14]
    old = _plain_logps(x, labels).float() + 0.05
    adv = torch.randn(14, generator=torch.Generator().manual_seed(1))
    w = torch.full((14,), 1 / 12)
    upstream = torch.randn(14, generator=torch.Generator().manual_seed(2))

    def plain(which):
        z = x.double().requires_grad_(True)
        logp = _plain_logps(z, labels, 0.9)
        if which == "logps":
            loss = (logp * upstream.double()).sum()
        elif which == "preference":
            S = [logp[a:b].sum() for a, b in zip(cu, cu[1:])]
            loss = torch.stack([-torch.nn.functional.logsigmoid(0.1 * (S[p] - S[2 + p])) for p in range(2)]).mean()
        else:
            r = (logp - old.double()).exp()
            pg = -torch.minimum(r * adv, r.clamp(0.8, 1.2) * adv)
            gap = old.double() - logp
            loss = ((pg + 0.1 * (torch.expm1(gap) - gap)) * w)[labels >= 0].sum()
        (d,) = torch.autograd.grad(loss * factor, z)
        return float(loss.detach()), d

    for which in ("logps", "preference", "policy"):
        z = x.to(DEV).requires_grad_(True)
        lab, dev = labels.to(DEV), lambda t: t.to(DEV)
        if which == "logps":
            loss = (torch_ops.token_logps(z, lab, 0.9) * dev(upstream)).sum()
        elif which == "preference":
            loss = torch_ops.preference_loss(z, lab, torch.tensor(cu, dtype=torch.int32, device=DEV), beta=0.1,
                                             temperature=0.9)[0]
        else:
            loss = torch_ops.policy_loss(z, lab, dev(old), dev(adv), dev(w), ref_logps=dev(old), kl_beta=0.1,
                                         temperature=0.9)[0]
        value, want = plain(which)
        assert abs(float(loss.detach()) - value) <= 1e-5 * max(1, abs(value))
        (loss * factor).backward(retain_graph=which != "logps")
        _close(z.grad, want, TOL[dtype])
        if which != "logps":
            with pytest.raises(RuntimeError, match="once"):
                loss.backward()


@pytest.mark.gpu
def test_opcheck():
    x, labels = _inputs(torch.float32)
    x, labels = x.to(DEV), labels.to(DEV)
    cu = torch.tensor([0, 4, 7, 11, 14], dtype=torch.int32, device=DEV)
    adv = torch.ones(14, device=DEV)
    check = lambda op, args: torch.library.opcheck(op, args, test_utils=("test_schema", "test_faketensor"))  # noqa: E731
    check(torch.ops.lora_gb300.token_logps, (x, labels, 1.0))
    check(torch.ops.lora_gb300.preference_loss, (x, labels, cu, None, 0.1, "hinge", 0.0, False, 1.0, True))
    check(torch.ops.lora_gb300.policy_loss, (x, labels, None, adv, None, None, 0.2, 0.2, 0.0, 1.0, True))


@pytest.mark.gpu
def test_without_gradient_and_in_inference():
    x, labels = _inputs(torch.bfloat16)
    x, labels = x.to(DEV), labels.to(DEV)
    with torch.no_grad():
        loss, pair, seq = torch_ops.preference_loss(x, labels, torch.tensor([0, 7, 14], dtype=torch.int32, device=DEV))
    assert not loss.requires_grad and pair.shape == (1,) and seq.shape == (2,)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_follows_torch(bits):
    """Twenty steps beside torch.optim.AdamW in fp32: 32-bit states agree to fp32 rounding; 8-bit
    states carry e4m3's 2^-4 of each state, so the parameters stay within 10 % of the way gone."""
    g = torch.Generator().manual_seed(0)
    start = [torch.randn(33, 70, generator=g), torch.randn(513, generator=g), torch.randn(4, 4, generator=g)]
    mine = [t.clone().to(DEV).requires_grad_() for t in start]
    ref = [t.clone().to(DEV).requires_grad_() for t in start]
    a = torch_ops.AdamW(mine, lr=1e-2, weight_decay=0.05, state_bits=bits)
    b = torch.optim.AdamW(ref, lr=1e-2, weight_decay=0.05)
    for step in range(20):
        for i, (p, q) in enumerate(zip(mine, ref)):
            p.grad = (torch.randn(p.shape, generator=g) + 0.5).to(DEV)
            q.grad = p.grad.clone()
        a.step()
        b.step()
    for p, q, s in zip(mine, ref, start):
        off, way = (p - q).detach().norm(), (q.detach() - s.to(DEV)).norm()
        assert float(off) <= (1e-5 if bits == 32 else 0.1) * float(way)
    # a parameter without a gradient stays; clipping reports the norm
    mine[2].grad = None
    before = mine[2].detach().clone()
    c = torch_ops.AdamW(mine, lr=1e-2, max_norm=0.5, state_bits=bits)
    c.step()
    assert torch.equal(mine[2].detach(), before)
    want = math.sqrt(sum(float(p.grad.double().square().sum()) for p in mine[:2]))
    assert abs(float(c.norm[0]) - want) <= 1e-5 * want and abs(float(c.norm[1]) - 0.5 / want) < 1e-5
    with pytest.raises(ValueError):
        torch_ops.AdamW(mine, state_bits=16)


@pytest.mark.gpu
@pytest.mark.parametrize("bits,masters", [(32, False), (8, True)])
def test_optimizer_resumes_and_takes_other_layouts(bits, masters):
    g = torch.Generator().manual_seed(0)
    start = [torch.randn(40, 30, generator=g).bfloat16(), torch.randn(300, generator=g).bfloat16()]
    grads = [[torch.randn(p.shape, generator=g) for p in start] for _ in range(4)]
    make = lambda values: [t.detach().clone().to(DEV).requires_grad_() for t in values]  # noqa: E731

    def run(params, opt, steps, transpose=False):
        for step in steps:
            for p, v in zip(params, grads[step]):
                v = v.bfloat16().to(DEV)
                p.grad = v.t().contiguous().t() if transpose and v.dim() == 2 else v
            opt.step()

    options = dict(lr=1e-2, state_bits=bits, masters=masters, max_norm=1.0)
    a = make(start)
    opt_a = torch_ops.AdamW(a, **options)
    run(a, opt_a, range(4))
    b = make(start)
    opt_b = torch_ops.AdamW(b, **options)
    run(b, opt_b, range(2), transpose=True)
    state = opt_b.state_dict()
    c = make(b)
    opt_c = torch_ops.AdamW(c, **options)
    opt_c.load_state_dict(state)
    run(c, opt_c, range(2, 4))
    for p, q in zip(a, c):
        assert torch.equal(p, q)
    for k, v in opt_a.state_dict().items():
        w = opt_c.state_dict()[k]
        same = lambda t, u: torch.equal(t.view(torch.uint8), u.view(torch.uint8))  # noqa: E731
        assert v == w if k == "step" else all(same(t, u) for t, u in zip(v, w)), k
    with pytest.raises(ValueError):
        torch_ops.AdamW(make(start), lr=1e-2, state_bits=40 - bits).load_state_dict(state)


@pytest.mark.gpu
@pytest.mark.parametrize("args", [["--loss", "preference", "--state-bits", "8"],
                                  ["--loss", "policy", "--state-bits", "32"]])
def test_example_learns(args):
    spec = importlib.util.spec_from_file_location("preference_finetune",
                                                  os.path.join(ROOT, "examples", "preference_finetune.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.main(args + ["--steps", "30"])
    assert all(math.isfinite(v) for v in losses)
    if "preference" in args:
        assert abs(losses[0] - math.log(2)) < 1e-3 and losses[-1] < 0.8 * losses[0]
    else:
        assert losses[-1] < losses[0] - 0.01
