"""The AdamW step over many tensors and the gradient norm against plain implementations.

States in 32 bits: against the formula in 64 bits; m and v carry a few roundings of
2^-24 of their terms, p those of the update (m, u, the quotient: some 8 of 2^-24 of
lr * |m / u|) and of itself.  States in 8 bits: the codes and scales follow single
IEEE roundings, so they are compared bit for bit with the same steps in torch."""
import math

import pytest
import torch

from lora_rank_adapter_gb300 import _build
from lora_rank_adapter_gb300 import training

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 0, 5000, 40000]


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)


def blocks(x):
    """[n] -> [blocks, 256], zeros past the end."""
    n = -(-x.numel() // 256) * 256
    return torch.nn.functional.pad(x.reshape(-1), (0, n - x.numel())).view(-1, 256)


def quantize(x, least=0.0):
    top = blocks(x).abs().amax(1)
    top = torch.where(top.isnan(), top, top.clamp(min=1e-30))
    q = blocks(x) * torch.div(torch.full_like(top, 448.0), top)[:, None]
    if least:
        q = torch.where(blocks(x) > 0, torch.where(q.isnan(), q, q.clamp(min=least)), q)
    return q.to(E4M3).view(-1)[:x.numel()], top * (1 / 448.0)


def dequantize(q, scale):
    return (blocks(q.float()) * scale[:, None]).view(-1)[:q.numel()]


def view(values, offset, dtype):
    """The values inside a larger buffer of sentinels, `offset` elements in."""
    full = torch.full((values.numel() + offset + 9,), 3, dtype=torch.float32).to(dtype).to(DEV)
    t = full[offset:offset + values.numel()]
    t.copy_(values.to(dtype))
    return full, t


def make(sizes, param, grad, bits, master, offset=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    s = {k: [] for k in ("p", "g", "m", "v", "ms", "vs", "w", "all")}
    for n in sizes:
        value = torch.randn(n, generator=g) * 0.05
        grads = torch.randn(n, generator=g) * 1e-2 * torch.exp(2 * torch.randn(n, generator=g))
        m, u = torch.randn(n, generator=g) * 1e-3, torch.rand(n, generator=g) * 1e-2
        if bits == 8:
            (mq, ms), (uq, us) = quantize(m), quantize(u, 2.0 ** -9)
        items = {"p": (value, param), "g": (grads, grad)}
        if master:
            items["w"] = (value, F32)
        if bits == 8:
            items.update(m=(mq.float(), E4M3), v=(uq.float(), E4M3), ms=(ms, F32), vs=(us, F32))
        else:
            items.update(m=(m, F32), v=(u * u, F32))
        for k, (v, dt) in items.items():
            full, t = view(v, offset, dt)
            s[k].append(t)
            s["all"].append((full, offset, t.numel()))
    s["plan"] = training.lora_adamw_plan(s["p"], s["g"], s["m"], s["v"], masters=s["w"] or None,
                                         exp_avg_scales=s["ms"] or None, exp_avg_sq_scales=s["vs"] or None)
    return s


def cpu(s):
    return {k: [t.detach().cpu().clone() for t in s[k]] for k in ("p", "g", "m", "v", "ms", "vs", "w")}


def sentinels_hold(s):
    for full, o, n in s["all"]:
        rest = torch.cat([full[:o], full[o + n:]]).float()
        assert bool((rest == 3).all())


def check_step(before, after, i, step, factor, bits, master):
    b1, b2, lr = HYPER["beta1"], HYPER["beta2"], HYPER["lr"]
    g = before["g"][i].double() * factor
    if bits == 8:
        m, v = dequantize(before["m"][i], before["ms"][i]).double(), dequantize(before["v"][i], before["vs"][i]).double() ** 2
    else:
        m, v = before["m"][i].double(), before["v"][i].double()
    m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    denom = (v / (1 - b2 ** step)).sqrt() + HYPER["eps"]
    p = (before["w"] if master else before["p"])[i].double()
    upd = lr / (1 - b1 ** step) * m / denom
    want = p * (1 - lr * HYPER["weight_decay"]) - upd
    tol = 2.0 ** -22 * want.abs() + 2.0 ** -20 * (upd.abs() + lr * (1 - b1) * g.abs() / denom / (1 - b1 ** step)) + 1e-12
    got = (after["w"] if master else after["p"])[i].double()
    if master:
        assert torch.equal(after["w"][i].to(after["p"][i].dtype), after["p"][i])
    elif after["p"][i].dtype == BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    assert bool(((got - want).abs() <= tol).all())
    if bits == 32:
        assert bool(((after["m"][i].double() - m).abs() <= 2.0 ** -21 * (before["m"][i].double().abs() + g.abs())).all())
        assert bool(((after["v"][i].double() - v).abs() <= 2.0 ** -21 * v.abs() + 1e-38).all())


def codes_equal(after, before, i, factor):
    """The 8-bit states by the same single roundings in torch, bit for bit."""
    f = torch.tensor(factor, dtype=F32)
    g = before["g"][i].float() * f
    m = dequantize(before["m"][i], before["ms"][i])
    u = dequantize(before["v"][i], before["vs"][i])
    m = m * HYPER["beta1"] + g * (1 - HYPER["beta1"])
    v = (u * u) * HYPER["beta2"] + (g * g) * (1 - HYPER["beta2"])
    for q, scale, x, least in (("m", "ms", m, 0.0), ("v", "vs", v.sqrt(), 2.0 ** -9)):
        want_q, want_s = quantize(x, least)
        assert torch.equal(after[q][i].view(torch.uint8), want_q.view(torch.uint8)), q
        assert torch.equal(after[scale][i].isnan(), want_s.isnan()), scale
        assert torch.equal(after[scale][i].nan_to_num(), want_s.nan_to_num()), scale


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", [(F32, F32, False), (BF16, F32, True), (BF16, BF16, False),
                                               (F32, BF16, False), (BF16, BF16, True)])
@pytest.mark.parametrize("offset", [0, 3, 8])
def test_adamw(bits, param, grad, master, offset):
    s = make(SIZES, param, grad, bits, master, offset)
    factor = 0.37
    f = torch.full((1,), factor, device=DEV)
    for step in (1, 2, 50):
        before = cpu(s)
        training.lora_adamw(s["plan"], step=step, grad_factor=f, **HYPER)
        after = cpu(s)
        for i, n in enumerate(SIZES):
            check_step(before, after, i, step, float(f), bits, master)
            assert torch.equal(before["g"][i], after["g"][i])
            if bits == 8:
                codes_equal(after, before, i, factor)
    sentinels_hold(s)


def test_many_tensors_and_no_factor():
    """More tensors than one launch of the layout takes, of very different sizes."""
    sizes = [1 + (i * 977) % 5003 for i in range(600)]
    s = make(sizes, F32, F32, 32, False)
    before = cpu(s)
    training.lora_adamw(s["plan"], step=4, **HYPER)
    after = cpu(s)
    for i in range(600):
        check_step(before, after, i, 4, 1.0, 32, False)
    sentinels_hold(s)


def test_transposed_and_matrix_parameters():
    """Any dense layout that the tensors of one parameter share."""
    g = torch.Generator().manual_seed(3)
    base = {k: torch.randn(48, 30, generator=g) for k in "pgmv"}
    base["v"] = base["v"].abs()
    a = {k: t.to(DEV).clone() for k, t in base.items()}
    b = {k: t.to(DEV).t().contiguous().t() for k, t in base.items()}
    for s in (a, b):
        plan = training.lora_adamw_plan([s["p"]], [s["g"]], [s["m"]], [s["v"]])
        training.lora_adamw(plan, step=1, **HYPER)
    for k in "pmv":
        assert torch.equal(a[k], b[k]), k
    with pytest.raises(ValueError):
        training.lora_adamw_plan([a["p"]], [b["g"]], [a["m"]], [a["v"]])
    with pytest.raises(ValueError):
        training.lora_adamw_plan([a["p"][:, :5]], [a["g"][:, :5]], [a["m"][:, :5]], [a["v"][:, :5]])
    with pytest.raises(ValueError):
        training.lora_adamw_plan([a["p"]], [a["g"]], [a["m"].bfloat16()], [a["v"]])
    with pytest.raises(TypeError):
        training.lora_adamw_plan([a["p"].half()], [a["g"]], [a["m"]], [a["v"]])


def test_eight_bit_states_keep_small_roots_zeros_and_nan():
    n = 1024
    s = make([n], F32, F32, 8, False)
    g = torch.zeros(n)
    g[0], g[1] = 1.0, 1e-7                 # block 0: a root 1e-7 of the largest would round to zero
    g[300] = math.nan                      # block 1
    g[512:768] = 1e-33                     # block 2: below the least magnitude of a scale
    s["g"][0].copy_(g)
    for k in ("m", "v", "ms", "vs"):
        s[k][0].view(torch.uint8 if k in "mv" else F32).zero_()
    before = cpu(s)
    training.lora_adamw(s["plan"], step=1, **HYPER)
    after = cpu(s)
    codes_equal(after, before, 0, 1.0)
    u = dequantize(after["v"][0], after["vs"][0])
    assert float(u[1]) > 0 and float(u[2]) == 0
    p = after["p"][0]
    assert bool(p[:256].isfinite().all()) and math.isnan(float(p[300])) and bool(p[512:].isfinite().all())
    assert bool(after["ms"][0][1].isnan()) and bool(after["ms"][0][[0, 2, 3]].isfinite().all())
    # the small root keeps the second step small: |update| stays within a few lr
    s["g"][0].zero_()
    p0 = s["p"][0].clone()
    training.lora_adamw(s["plan"], step=2, **HYPER)
    assert float((s["p"][0] - p0)[:256].abs().max()) < 20 * HYPER["lr"]


@pytest.mark.parametrize("grad", [F32, BF16])
@pytest.mark.parametrize("sizes,offset", [([1], 0), (SIZES, 0), (SIZES, 3), ([100000, 3, 70001], 1), ([0], 0), ([], 0)])
def test_grad_norm(grad, sizes, offset):
    """The norm sums squares in fp32 over 8 elements and in 64 bits beyond: 2^-21 relative."""
    s = make(sizes, F32, grad, 32, False, offset)
    want = math.sqrt(sum(float((t.double() ** 2).sum()) for t in s["g"]))
    out = torch.full((2,), 9.0, device=DEV)
    for limit in (0.5 * want, 2 * want + 1, 0.0):
        training.lora_grad_norm(s["plan"], limit, out)
        norm, factor = (float(v) for v in out)
        assert abs(norm - want) <= 2.0 ** -21 * want
        assert abs(factor - min(1.0, limit / (want + 1e-6))) <= 2.0 ** -20
    again = torch.empty(2, device=DEV)
    training.lora_grad_norm(s["plan"], 0.0, again)
    assert torch.equal(out, again)
    if sizes and sizes[0]:
        s["g"][0][0] = math.nan
        training.lora_grad_norm(s["plan"], 1.0, out)
        assert bool(out.isnan().all())
        s["g"][0][0] = math.inf
        training.lora_grad_norm(s["plan"], 1.0, out)
        assert float(out[0]) == math.inf and float(out[1]) == 0
